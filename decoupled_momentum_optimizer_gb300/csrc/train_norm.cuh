// What the root-mean-square norm and its gradient share: how a row lies in registers.
#pragma once

#include "train_pairs.cuh"

namespace demo {

// ----------------------------------------------------------------------------
// A row in registers
// ----------------------------------------------------------------------------

// A warp holds `per` units of 32 N consecutive columns of a row; in a unit, lane l holds N consecutive ones as
// one 16-byte access, or, where rows are not whole aligned accesses, N columns 32 apart (N = 4, so that a block
// of 128 is one unit of one warp).  Rows of less than a unit are held by `lanes` lanes, a power of two, and a
// warp holds 32 / lanes of them.  A lane's pointers go to its first column, so that unit j is at a constant
// offset, and one comparison per unit says whether it is in the row.
template <typename T, bool VEC>
constexpr int kNormN = VEC ? 16 / static_cast<int>(sizeof(T)) : 4;

struct Place {
  int first;  // column of the lane's first element
  int reach;  // columns of the warp from there on; 0 or less where it has none
  int lanes;
  template <bool VEC, int N>
  __device__ __forceinline__ static Place of(int warp, int per, int lane, int lanes, int cols) {
    const int begin = warp * per * 32 * N, mine = cols - begin < per * 32 * N ? cols - begin : per * 32 * N;
    const int at = VEC ? lane * N : lane;
    return Place{begin + at, mine - at, lanes};
  }
  // Whether the warp has columns in unit j (the same for all of its lanes), lane being the lane in its row.
  template <bool VEC, int N>
  __device__ __forceinline__ bool unit(int j, int lane) const {
    return reach + (VEC ? lane * N : lane) > j * 32 * N;
  }
  // Offset of element e of unit j from the lane's first, and whether it is in the row.
  template <bool VEC, int N>
  __device__ __forceinline__ int offset(int j, int e) const {
    return j * 32 * N + (VEC ? e : lanes * e);
  }
  template <bool VEC, int N>
  __device__ __forceinline__ bool has(int j, int e) const {
    return offset<VEC, N>(j, VEC ? 0 : e) < reach;
  }
};

// Sums and magnitudes of packed elements.  The sum of two 16-bit values rounded once is their float32 sum
// rounded: 24 bits are at least 2 * 11 + 2.
template <typename T>
__device__ __forceinline__ uint32_t packed_add(uint32_t a, uint32_t b) {
  using V = std::conditional_t<is_bf16<T>, __nv_bfloat162, __half2>;
  const V r = __hadd2_rn(*reinterpret_cast<const V*>(&a), *reinterpret_cast<const V*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T>
__device__ __forceinline__ uint32_t packed_max_abs(uint32_t m, uint32_t a) {
  using V = std::conditional_t<is_bf16<T>, __nv_bfloat162, __half2>;
  const V r = __hmax2(*reinterpret_cast<const V*>(&m), __habs2(*reinterpret_cast<const V*>(&a)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// A lane's N elements of a unit: 16 bits stay packed in words (as an array of 16-bit elements they took a
// register each), float32 is itself.
template <typename T, bool VEC, int N>
struct Unit {
  static constexpr bool kPacked = sizeof(T) == 2;
  static constexpr int kWords = kPacked ? N / 2 : N;
  uint32_t w[kWords];

  // Elements 2 i and 2 i + 1.
  __device__ __forceinline__ F2 get2(int i) const {
    if constexpr (kPacked) return widen<T>(w[i]);
    return f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
  }
  // Their float32 values rounded to T.
  __device__ __forceinline__ void set2(int i, F2 v) {
    if constexpr (kPacked) {
      w[i] = narrow<T>(v);
    } else {
      w[2 * i] = __float_as_uint(v.x);
      w[2 * i + 1] = __float_as_uint(v.y);
    }
  }
  __device__ __forceinline__ void add(const Unit& o) {
#pragma unroll
    for (int i = 0; i < (kPacked ? kWords : N / 2); ++i) {
      if constexpr (kPacked)
        w[i] = packed_add<T>(w[i], o.w[i]);
      else
        set2(i, add2(get2(i), o.get2(i)));
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // The lane's elements of unit j, zero past the row's end.  CONST: memory that the kernel does not write.
  template <bool CONST = false>
  __device__ __forceinline__ void load(const T* p, const Place& at, int j) {
    if constexpr (VEC) {
      if (at.has<VEC, N>(j, 0)) {
        const uint4* q = reinterpret_cast<const uint4*>(p + at.offset<VEC, N>(j, 0));
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
          const uint4 v = CONST ? __ldg(q + i) : q[i];
          w[4 * i] = v.x;
          w[4 * i + 1] = v.y;
          w[4 * i + 2] = v.z;
          w[4 * i + 3] = v.w;
        }
      } else {
        clear();
      }
    } else {
      using Bits = std::conditional_t<kPacked, uint16_t, uint32_t>;
      Bits b[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        b[e] = 0;
        if (at.has<VEC, N>(j, e)) {
          const Bits* q = reinterpret_cast<const Bits*>(p + at.offset<VEC, N>(j, e));
          b[e] = CONST ? __ldg(q) : *q;
        }
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = kPacked ? b[2 * i] | static_cast<uint32_t>(b[2 * i + 1]) << 16 : b[i];
    }
  }
  __device__ __forceinline__ void store(T* p, const Place& at, int j) const {
    if constexpr (VEC) {
      if (at.has<VEC, N>(j, 0)) *reinterpret_cast<uint4*>(p + at.offset<VEC, N>(j, 0)) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (at.has<VEC, N>(j, e)) {
          if constexpr (kPacked)
            reinterpret_cast<uint16_t*>(p)[at.offset<VEC, N>(j, e)] = static_cast<uint16_t>(e % 2 ? w[e / 2] >> 16 : w[e / 2]);
          else
            reinterpret_cast<uint32_t*>(p)[at.offset<VEC, N>(j, e)] = w[e];
        }
      }
    }
  }
};

template <typename V>
__device__ __forceinline__ V lane_sum(V v, int lanes = 32) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    if (d < lanes) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// Host: whether rows are whole 16-byte accesses of n elements.
inline bool whole_rows(const void* q, long long ld, int n) {
  return (reinterpret_cast<uintptr_t>(q) & 15) == 0 && ld % n == 0;
}

// Host: lanes of a row of `accesses` accesses, the next power of two.
inline int row_lanes(long long accesses) {
  int l = 1;
  while (l < 32 && l < accesses) l *= 2;
  return l;
}

}  // namespace demo
