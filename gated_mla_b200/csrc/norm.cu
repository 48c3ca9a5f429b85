// norm.cu — the residual's addition and the root-mean-square norm in front of a
// layer, with an optional E4M3 output.
//
//   s = x + r (fp32; s = x without a residual)          residual_out = s
//   y = s / sqrt(mean(s^2) + eps) * w                    out = y
//   codes = E4M3(y / scale_g), scale_g = max |y| over the group / 448 (1 for a group of zeros)
//
// Sums, the norm and the scale stay in fp32; s and y are rounded once, when they
// are stored, and y is formed from the unrounded s.
//
// Bound by HBM: each element is read and written once (16384 rows of 7168 with a residual: 162 us, 0.90
// of the rate of a copy; with codes as well 227 us, 0.72: eight divisions and a group maximum for each
// vector show). A row is held in
// registers between the two passes (mean, then scaling), 8 consecutive elements a
// thread and vector, so a group of 32 .. 256 elements is 4 .. 32 neighbouring
// lanes and its maximum needs shuffles only.
#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gmla {

namespace {

template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, bool vec, float (&v)[8]);

template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, int n, bool vec, float (&v)[8]) {
  if (vec) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.f;
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, int n, bool vec, float (&v)[8]) {
  if (vec) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
  }
}

__device__ __forceinline__ void store8(__nv_bfloat16* p, int n, bool vec, const float (&v)[8]) {
  if (vec) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                              pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = __float2bfloat16_rn(v[i]);
  }
}
__device__ __forceinline__ void store8(float* p, int n, bool vec, const float (&v)[8]) {
  if (vec) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}

// Registers a thread. The bf16 forms wait for HBM with their loads in flight, so rows resident count
// for more than the few words spilled (16384 rows of 7168, four vectors: 161 us with 56 registers, 165
// with 52, 176 with 64; of 4096, two vectors and no codes: 84 us with 32, 89 with 40, 109 with the
// weights loaded early and 64; of 2048, one vector: 47 us with 32, 53 with 40). fp32 rows have twice
// the bytes in flight.
// 1024 threads of 64 are what a block may hold.
constexpr int norm_regs(int vpt, bool f32, bool grp) {
  return f32 ? 64 : (vpt == 4 ? 56 : (vpt == 2 && grp ? 40 : 32));
}

}  // namespace

// One row per `warps` warps; VPT vectors of 8 elements a thread (vector i of lane t
// covers elements 8 (i * 32 * warps + t) ..). blockDim = warps * 32 * rows a block.
// VEC: d, the row strides and the addresses allow 16-byte accesses, and every vector is whole.
template <typename T, int VPT, bool VEC, bool GRP>
__global__ void __maxnreg__(norm_regs(VPT, sizeof(T) == 4, GRP)) add_rms_norm_kernel(NormArgs a) {
  __shared__ float s_sum[32];
  griddep_wait();
  griddep_launch_dependents();
  const int tpr = a.warps * 32;
  const int lane_r = threadIdx.x % tpr;
  const int warp0 = threadIdx.x / tpr * a.warps;      // first warp of this row in the block
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  const bool live = row < a.T;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* r = static_cast<const T*>(a.residual) + row * a.residual_stride;
  T* ro = static_cast<T*>(a.residual_out) + row * a.residual_out_stride;
  T* out = static_cast<T*>(a.out) + row * a.out_stride;
  const T* wt = static_cast<const T*>(a.weight);
  float v[VPT][8], w8[VPT][8];
  // every load of the row, then, in the form for few rows, the weights (held for after the reduction)
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = (i * tpr + lane_r) * 8;
    const int n = live ? min(8, a.d - e) : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (n > 0) load8<T>(x + e, n, VEC, v[i]);
  }
  if (a.residual) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int e = (i * tpr + lane_r) * 8;
      const int n = live ? min(8, a.d - e) : 0;
      float u[8];
      if (n > 0) {
        load8<T>(r + e, n, VEC, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] += u[j];
      }
    }
  }
  if (VPT == 1 && wt) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int e = (i * tpr + lane_r) * 8;
      const int n = live ? min(8, a.d - e) : 0;
      if (n > 0) load8<T>(wt + e, n, VEC, w8[i]);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = (i * tpr + lane_r) * 8;
    const int n = live ? min(8, a.d - e) : 0;
    if (n > 0 && a.residual_out) store8(ro + e, n, VEC, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(v[i][j], v[i][j], sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (a.warps > 1) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) s_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = lane < a.warps ? s_sum[warp0 + lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
  const float inv = rsqrtf(sum / static_cast<float>(a.d) + a.eps);
  const int g8 = a.group >> 3;           // lanes a group spans
  const int n_group = GRP ? (a.d + a.group - 1) / a.group : 0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int e = (i * tpr + lane_r) * 8;
    const int n = live ? min(8, a.d - e) : 0;
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = v[i][j] * inv;
    if (n > 0 && wt) {
      if (VPT > 1) load8<T>(wt + e, n, VEC, w8[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] *= w8[i][j];
    }
    if (n > 0 && a.out) store8(out + e, n, VEC, y);
    if (GRP) {
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, VEC || j < n ? fabsf(y[j]) : 0.f);
      if (n <= 0) top = 0.f;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
        if (o < g8) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (n > 0) {
        const float part = top / 448.f;              // 0 for a group of zeros (or of values too small to divide)
        const float scale = part > 0.f ? part : 1.f;
        if ((threadIdx.x & (g8 - 1)) == 0) a.scales[row * n_group + e / a.group] = scale;
        uint8_t* c = a.codes + row * a.d + e;
        // a true division: next to a rounding border a reciprocal's error picks another code
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = y[j] / scale;
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = __nv_cvt_float2_to_fp8x2(make_float2(y[4 * h], y[4 * h + 1]), __NV_SATFINITE, __NV_E4M3) |
                 (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(y[4 * h + 2], y[4 * h + 3]),
                                                                 __NV_SATFINITE, __NV_E4M3))
                  << 16);
        if (VEC) {
          *reinterpret_cast<uint2*>(c) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < n) c[j] = static_cast<uint8_t>(w[j >> 2] >> (8 * (j & 3)));
        }
      }
    }
  }
}

template <typename T, bool VEC, bool GRP>
static cudaError_t launch_norm(const NormArgs& a, int vpt, dim3 grid, dim3 block, cudaStream_t st) {
  switch (vpt) {
    case 1: return launch_pdl(add_rms_norm_kernel<T, 1, VEC, GRP>, grid, block, 0, st, 1, a);
    case 2: return launch_pdl(add_rms_norm_kernel<T, 2, VEC, GRP>, grid, block, 0, st, 1, a);
    default: return launch_pdl(add_rms_norm_kernel<T, 4, VEC, GRP>, grid, block, 0, st, 1, a);
  }
}

template <typename T>
static cudaError_t launch_norm_t(const NormArgs& a, int vpt, dim3 grid, dim3 block, cudaStream_t st) {
  if (a.vec) return a.group ? launch_norm<T, true, true>(a, vpt, grid, block, st) : launch_norm<T, true, false>(a, vpt, grid, block, st);
  return a.group ? launch_norm<T, false, true>(a, vpt, grid, block, st) : launch_norm<T, false, false>(a, vpt, grid, block, st);
}

cudaError_t launch_add_rms_norm(NormArgs a, bool f32, int num_sms, cudaStream_t st) {
  const int nvec = (a.d + 7) / 8;
  const int vpt = norm_vectors(a.d, a.T, f32, num_sms);
  a.warps = (nvec + 32 * vpt - 1) / (32 * vpt);
  const int rows = a.warps >= 8 ? 1 : 8 / a.warps;       // rows a block (256 threads or one row)
  const dim3 block(a.warps * 32 * rows);
  const dim3 grid((a.T + rows - 1) / rows);
  prof_begin(st, "add_rms_norm");
  cudaError_t e = f32 ? launch_norm_t<float>(a, vpt, grid, block, st) : launch_norm_t<__nv_bfloat16>(a, vpt, grid, block, st);
  prof_end(st);
  return e;
}

// Vectors a thread. Few rows: as few as 32 warps allow (the shortest chain: 8 rows of 7168
// take 2.6 us with one, 3.8 with four). Many: about 8 warps a row, so that an SM holds
// several rows in different phases (16384 rows of 7168: 161 us with four, 0.90 of the HBM
// rate, 167 with two, 188 with one; in fp32 293 with four, 274 with two).
int norm_vectors(int d, int T, bool f32, int num_sms) {
  const int nvec = (d + 7) / 8;
  if (T <= 2 * num_sms) return nvec <= 1024 ? 1 : (nvec <= 2048 ? 2 : 4);
  return nvec <= 256 ? 1 : (nvec <= (f32 ? 1024 : 512) ? 2 : 4);
}

}  // namespace gmla
