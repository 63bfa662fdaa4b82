// Element access shared by the kernels around the expert block: rows of
// bf16, fp16 or fp32 read and written in 16-byte vectors (or element by
// element where rows are not 16-byte aligned), always computed on in fp32.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"

namespace moe {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// Two fp32 values rounded to a packed pair of 16-bit ones.
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi, __nv_bfloat16) {
  return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi, __half) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_pair(uint32_t v, __nv_bfloat16) {
  return make_float2(bf16lo(v), bf16hi(v));
}
__device__ __forceinline__ float2 unpack_pair(uint32_t v, __half) {
  return __half22float2(*reinterpret_cast<__half2*>(&v));
}

// VEC elements of T as they lie in memory: a 16-byte vector, or one element.
template <typename T, int VEC>
struct Raw {
  static_assert(VEC * sizeof(T) == 16 || VEC == 1, "16 bytes or one element");
  static constexpr bool kVec = VEC > 1;
  using Store = typename std::conditional<kVec, uint4, T>::type;
  Store v;

  __device__ __forceinline__ void unpack(float (&f)[VEC]) const {
    if constexpr (!kVec) {
      f[0] = to_f32<T>(v);
    } else if constexpr (sizeof(T) == 4) {
      f[0] = __uint_as_float(v.x);
      f[1] = __uint_as_float(v.y);
      f[2] = __uint_as_float(v.z);
      f[3] = __uint_as_float(v.w);
    } else {
      const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = unpack_pair(q[i], T{});
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
      }
    }
  }
  __device__ __forceinline__ void pack(const float (&f)[VEC]) {
    if constexpr (!kVec) {
      v = from_f32<T>(f[0]);
    } else if constexpr (sizeof(T) == 4) {
      v = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                     __float_as_uint(f[3]));
    } else {
      uint32_t q[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) q[i] = pack_pair(f[2 * i], f[2 * i + 1], T{});
      v = make_uint4(q[0], q[1], q[2], q[3]);
    }
  }
  // zeros for the first e < VEC elements
  __device__ __forceinline__ void clear_below(int e) {
    static_assert(kVec, "a vector");
    constexpr int kPer = 4 / sizeof(T);  // elements of a word
    uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if ((i + 1) * kPer <= e) q[i] = 0u;
      else if (kPer == 2 && 2 * i < e) q[i] &= 0xffff0000u;
    }
    v = make_uint4(q[0], q[1], q[2], q[3]);
  }
  // element i * VEC of a row
  __device__ __forceinline__ void load(const T* row, int i) {
    if constexpr (kVec) v = __ldcs(reinterpret_cast<const uint4*>(row) + i);
    else v = row[i];
  }
  __device__ __forceinline__ void store(T* row, int i) const {
    if constexpr (kVec) reinterpret_cast<uint4*>(row)[i] = v;
    else row[i] = v;
  }
};

// Two fp32 values that are computed on together (packed fp32 instructions take
// one issue slot for two operations), or one, under the same names.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 make_f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split(F2 a) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(a.v));
  return f;
}
__device__ __forceinline__ F2 fadd(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fmul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 ffma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float fadd(float a, float b) { return a + b; }
__device__ __forceinline__ float fmul(float a, float b) { return a * b; }
__device__ __forceinline__ float ffma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float fold(F2 a) {
  const float2 f = split(a);
  return f.x + f.y;
}
__device__ __forceinline__ float fold(float a) { return a; }

// VEC fp32 values as kN of those.
template <int VEC>
struct Nums {
  static constexpr int kN = VEC == 1 ? 1 : VEC / 2;
  using F = typename std::conditional<VEC == 1, float, F2>::type;
  static __device__ __forceinline__ F splat(float v) {
    if constexpr (VEC == 1) return v;
    else return make_f2(v, v);
  }
  static __device__ __forceinline__ void gather(const float (&f)[VEC], F (&n)[kN]) {
    if constexpr (VEC == 1) {
      n[0] = f[0];
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) n[i] = make_f2(f[2 * i], f[2 * i + 1]);
    }
  }
  static __device__ __forceinline__ void scatter(const F (&n)[kN], float (&f)[VEC]) {
    if constexpr (VEC == 1) {
      f[0] = n[0];
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        const float2 q = split(n[i]);
        f[2 * i] = q.x;
        f[2 * i + 1] = q.y;
      }
    }
  }
};

// A kernel that a call launches behind another of its own may start before
// that one has ended (its launch and set-up overlap the other's end); it waits
// here before it touches global memory.  What the other wrote is read by
// ordinary loads: __ldg and const __restrict__ pointers allow the read-only
// path, which asks that the data stay unchanged for as long as the kernel is
// resident.  Returns at once in a kernel that was launched without the
// attribute.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The kernel behind this one may be launched once every block has come here.
__device__ __forceinline__ void let_next_launch() { asm volatile("griddepcontrol.launch_dependents;"); }

// VEC weights (fp32 or T) as fp32; VEC > 1 asks for 16-byte alignment of W.
template <typename W, int VEC>
__device__ __forceinline__ void load_weights(const W* w, int i, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = to_f32<W>(__ldg(w + i));
  } else if constexpr (sizeof(W) == 4) {
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(w) + i * (VEC / 4) + q);
      f[4 * q] = a.x;
      f[4 * q + 1] = a.y;
      f[4 * q + 2] = a.z;
      f[4 * q + 3] = a.w;
    }
  } else {
    Raw<W, VEC> r;
    r.v = __ldg(reinterpret_cast<const uint4*>(w) + i);
    r.unpack(f);
  }
}

// 16 consecutive fp32 columns of the warp's 32 TMEM lanes (see tmem_ld_32x32b_x32).
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// 2^x to 2 ulp and 1 / x to 1 ulp, subnormals flushed.
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

}  // namespace moe
