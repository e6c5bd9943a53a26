// Device helpers shared by the block operators' kernels.
#pragma once
#include "block_internal.h"
#include "kernel_common.h"

namespace mq {

// The sequence a workgroup works on, from the device arrays, clamped to what
// the arrays hold: a wrong length or offset cannot lead outside them.
struct Seq {
  int q0;     // its first new token (row of q, k, v)
  int n;      // its new tokens
  int len;    // its tokens, the new ones counted
  int cap;    // those of them that the block table has room for
  int slot;   // its tail slot, -1 where the table names none that exists
};

// What no thread of the kernel writes: the load may be a scalar one, where the address is uniform, also in a loop that
// writes elsewhere.
template <typename T>
__device__ __forceinline__ T unwritten(const T* p) {
  return *(const __attribute__((address_space(4))) T*)p;
}

__device__ __forceinline__ Seq seq_of(const BatchView& b, const KvView& kv, int s) {
  Seq q;
  const int c0 = unwritten(b.cu + s), c1 = unwritten(b.cu + s + 1);
  q.q0 = min(max(c0, 0), b.tokens);
  q.n = min(max(c1, q.q0), b.tokens) - q.q0;
  q.len = max(unwritten(b.len + s), 0);
  q.cap = (int)min((int64_t)q.len, (int64_t)b.width * kKvBlock);
  const int slot = b.slot ? unwritten(b.slot + s) : s;
  q.slot = (unsigned)slot < (unsigned)kv.slots ? slot : -1;
  return q;
}

// v, as an fp32 value of its own: a conversion to fp16 behind it cannot be
// folded into the operation that made it, which would round once where the
// definition rounds twice, in some instances of a kernel and not in others.
__device__ __forceinline__ float fp32(float v) {
  asm("" : "+v"(v));
  return v;
}

// One pair turned: products and sums are rounded one by one (no fused
// multiply-add), so that the result is that of the formula in fp32 whatever
// the compiler does around it; a code of the cache then depends on the inputs
// alone.
__device__ __forceinline__ float2 turn(float a, float b, float2 cs) {
#pragma clang fp contract(off)
  const float ac = a * cs.x, bs = b * cs.y, bc = b * cs.x, as = a * cs.y;
  return make_float2(fp32(ac - bs), fp32(bc + as));
}

// (cos, sin) of pair i at position p; NaN outside the table.
__device__ __forceinline__ float2 cos_sin(const RopeView& r, int64_t p, int i) {
  if ((uint64_t)p >= (uint64_t)r.positions) return make_float2(__builtin_nanf(""), __builtin_nanf(""));
  return r.table[p * (r.rot >> 1) + i];
}

// Element d of a head row x, turned to position p.
__device__ __forceinline__ _Float16 turned(const _Float16* x, int d, const RopeView& r, int64_t p) {
  if (d >= r.rot) return x[d];
  const int half = r.rot >> 1;
  int a, b, i;
  if (r.interleaved) {
    i = d >> 1;
    a = d & ~1;
    b = a + 1;
  } else {
    i = d < half ? d : d - half;
    a = i;
    b = i + half;
  }
  const float2 y = turn((float)x[a], (float)x[b], cos_sin(r, p, i));
  return (_Float16)(d == a ? y.x : y.y);
}

// Eight fp16 values from or to any element of a tensor: one 16-byte access, which memory takes at any address.
typedef _Float16 half8_any_t __attribute__((ext_vector_type(8), aligned(2)));
typedef float float4_any_t __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ half8_t load8(const _Float16* p) { return *reinterpret_cast<const half8_any_t*>(p); }
__device__ __forceinline__ void store8(_Float16* p, const half8_t& v) { *reinterpret_cast<half8_any_t*>(p) = v; }

// Eight pairs (half layout: a the first elements, b the second ones) or four (interleaved: a) turned by the cosines and
// sines of NP pairs.
template <bool INTER, int NP>
__device__ __forceinline__ void turn_piece(half8_t& a, half8_t& b, const float2* cs) {
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const float2 r = INTER ? turn((float)a[2 * i], (float)a[2 * i + 1], cs[i]) : turn((float)a[i], (float)b[i], cs[i]);
    if (INTER) {
      a[2 * i] = (_Float16)r.x;
      a[2 * i + 1] = (_Float16)r.y;
    } else {
      a[i] = (_Float16)r.x;
      b[i] = (_Float16)r.y;
    }
  }
}

// (cos, sin) of NP pairs from pair i0 on at position p, the sines times dir; NaN outside the table.
template <int NP>
__device__ __forceinline__ void load_cos_sin(const RopeView& r, int64_t p, int i0, float dir, float2* cs) {
  if ((uint64_t)p < (uint64_t)r.positions) {
    const float4_any_t* row = reinterpret_cast<const float4_any_t*>(r.table + p * (r.rot >> 1) + i0);
#pragma unroll
    for (int i = 0; i < NP / 2; ++i) {
      const float4_t f = row[i];
      cs[2 * i] = make_float2(f.x, f.y * dir);
      cs[2 * i + 1] = make_float2(f.z, f.w * dir);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NP; ++i) cs[i] = make_float2(__builtin_nanf(""), __builtin_nanf(""));
  }
}

// Whether a rotation's pairs fall into pieces of 8 elements.
inline bool piecewise(const RopeView& r) { return r.rot % (r.interleaved ? 8 : 16) == 0; }

__device__ __forceinline__ bool finite_h(_Float16 v) {
  return (__builtin_bit_cast(uint16_t, v) & 0x7C00u) != 0x7C00u;
}

}  // namespace mq
