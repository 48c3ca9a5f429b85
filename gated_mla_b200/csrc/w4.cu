// w4.cu — the output product with 4-bit weights and group scales:
//
//   y[t, n] = sum_g scale[n, g] * sum_{k in group g} (code[n, k] - 8) * a[t, k],   a = gate ⊙ o
//
// codes: two per byte (even k in the low nibble), scale: bf16 per row and group of
// 32, 64 or 128 consecutive k.
//
// Few tokens (w4_mma): bound by the weights' N K / 2 bytes. A row tile's codes
// stream through a ring of TMA boxes (128 or 256 rows x 128 bytes = 256 k); the
// codes become bf16 in registers, straight into the A fragments of m16n8k16
// matrix instructions, and never return to shared memory (tcgen05 would need the
// expanded tile written there: 4 bytes of shared traffic for each byte of codes).
// A code v becomes the exact bf16 128 + v by one and-or on the packed word, minus
// 136; the products of one group are summed in fp32 and only then scaled, so no
// weight is ever rounded. One and-or takes nibbles i and i + 4 of a word, so
// the activations are stored with k, k + 4 side by side (w4_prep, which also
// applies the gate). K is split over the CTAs of a cluster, which add their fp32
// partial tiles through distributed shared memory in a fixed order.
//
// Many tokens: the codes expand once to bf16 (w4_expand: one rounding of
// (code - 8) * scale, 2^-9 relative) and the tcgen05 GEMM of the bf16 path runs.
#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gmla {

namespace {

constexpr int kW4Warps = 8;               // consumer warps; one more issues the copies
constexpr int kW4Threads = 32 * (kW4Warps + 1);
constexpr int kW4Chunk = 256;             // k per stage (128 bytes of codes a row)

__device__ __forceinline__ uint32_t w4_pair(uint32_t w, int i) {   // (128 + v_i, 128 + v_{i+4}) - 136 as bf16x2
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(r) : "r"(w >> (4 * i)));
  asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(0x43084308u));
  return r;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// Byte offset of 16-byte chunk `c` of row `r` in a box of 128-byte rows with the 128-byte swizzle.
__device__ __forceinline__ uint32_t sw128_chunk(uint32_t r, uint32_t c) { return r * 128u + ((c ^ (r & 7u)) << 4); }

struct W4Smem {
  uint64_t full[8], empty[8];
  int abort;
};

template <int NT, int MT>
struct W4Cfg {
  static constexpr int kRows = 16 * MT * kW4Warps;             // weight rows per CTA
  static constexpr int kWBytes = kRows * 128;
  static constexpr int kXBox = 8 * NT * 128;                   // [8 NT tokens x 64 k]
  static constexpr int kXBytes = kXBox * (kW4Chunk / 64);
  static constexpr int kStage = kWBytes + kXBytes;
  static constexpr int kStages = NT == 1 ? 5 : (NT == 2 ? 4 : 3);
  static constexpr int kRed = kRows * 8 * NT * 4;              // fp32 partial tile, over the ring once it has drained
  static constexpr int kRing = kStage * kStages > kRed ? kStage * kStages : kRed;
  static constexpr int kSmem = kRing + 1024 + static_cast<int>(sizeof(W4Smem));
  static_assert(kStages <= 8, "barriers");
  static_assert(kSmem <= 232448, "shared memory");
};

}  // namespace

// ---------------------------------------------------------------------------
// a = gate ⊙ o in bf16, each run of 8 stored as k 0 4 1 5 2 6 3 7
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) w4_prep_kernel(W4PrepArgs a) {
  griddep_wait();
  griddep_launch_dependents();   // all earlier kernels are done: the product may begin to load its weights
  const int k8 = a.K >> 3;
  const int64_t n = static_cast<int64_t>(a.T) * k8;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t t = i / k8;
    const int k = static_cast<int>(i - t * k8) * 8;
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.o) + t * a.K + k);
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if (a.gate_logits) {
      float g[8];
      if (a.gate_mode == kGateChannel) {
        const float4* z = reinterpret_cast<const float4*>(a.gate_logits + t * a.K + k);
        const float4 z0 = z[0], z1 = z[1];
        const float zz[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = 1.f / (1.f + expf(-zz[j]));
      } else {   // d_h is a multiple of 8: one head for the run
        const float gv = head_gate(a.gate_logits + t * a.H, a.H, k / a.d_h, a.gate_mode, a.gate_topk);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] = gv;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = pack_bf16x2(__uint_as_float(w[j] << 16) * g[2 * j], __uint_as_float(w[j] & 0xffff0000u) * g[2 * j + 1]);
    }
    uint4 r;
    r.x = __byte_perm(w[0], w[2], 0x5410);
    r.y = __byte_perm(w[0], w[2], 0x7632);
    r.z = __byte_perm(w[1], w[3], 0x5410);
    r.w = __byte_perm(w[1], w[3], 0x7632);
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + t * a.K + k) = r;
  }
}

// ---------------------------------------------------------------------------
// few tokens. Grid (row tiles, tiles of 8 NT tokens, K splits); the splits of a
// tile form a cluster. GPC groups per 256-k chunk (8, 4 or 2).
// ---------------------------------------------------------------------------
template <int NT, int MT, int GPC>
__global__ void __launch_bounds__(kW4Threads) w4_mma_kernel(const __grid_constant__ W4Args a) {
  using C = W4Cfg<NT, MT>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  W4Smem* sm = reinterpret_cast<W4Smem*>(ring + C::kRing);
  volatile int* abort_flag = &sm->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = gridDim.z, rank = blockIdx.z;
  const int n_chunk = (a.K + kW4Chunk - 1) / kW4Chunk;
  const int c_lo = static_cast<int>(static_cast<int64_t>(n_chunk) * rank / splits);
  const int c_hi = static_cast<int>(static_cast<int64_t>(n_chunk) * (rank + 1) / splits);
  const int row0 = blockIdx.x * C::kRows, t0 = blockIdx.y * 8 * NT;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sm->full[i], 1);
      mbar_init(&sm->empty[i], kW4Warps);
    }
    sm->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x == 0) griddep_launch_dependents();

  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[m][n][j] = 0.f;

  int issued = 0;   // stages requested (copy thread)
  if (warp == kW4Warps) {
    if (lane == 0) {
      // the weights: w4_prep, the kernel before this one, neither writes them nor starts
      // this one before all earlier kernels are done, so they are requested before the wait
      tma_prefetch_desc(&a.wmap);
      tma_prefetch_desc(&a.xmap);
      const uint64_t pol_w = l2_evict_first(), pol_x = l2_evict_last();
      const int n_c = c_hi - c_lo;
      int pre = n_c < NS ? n_c : NS;
      auto load_w = [&](int i) {
        const int s = i % NS;
        mbar_arrive_expect_tx(&sm->full[s], C::kStage);
        tma_load_2d(&a.wmap, &sm->full[s], ring + s * C::kStage, (c_lo + i) * 128, row0, pol_w);
      };
      auto load_x = [&](int i) {
        const int s = i % NS;
#pragma unroll
        for (int j = 0; j < kW4Chunk / 64; ++j)
          tma_load_2d(&a.xmap, &sm->full[s], ring + s * C::kStage + C::kWBytes + j * C::kXBox,
                      (c_lo + i) * kW4Chunk + j * 64, t0, pol_x);
      };
      for (int i = 0; i < pre; ++i) load_w(i);
      griddep_wait();
      for (int i = 0; i < pre; ++i) load_x(i);
      for (issued = pre; issued < n_c; ++issued) {
        if (!mbar_wait(&sm->empty[issued % NS], ((issued / NS) & 1) ^ 1, abort_flag, a.status)) break;
        load_w(issued);
        load_x(issued);
      }
    }
    __syncwarp();
  } else {
    const int g = lane >> 2, c = lane & 3;
    const int n_groups = a.K / a.group;
    const __nv_bfloat16* sc[MT][2];
    bool row_ok[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = row0 + (warp * MT + m) * 16 + g + 8 * h;
        row_ok[m][h] = row < a.N;
        sc[m][h] = static_cast<const __nv_bfloat16*>(a.scales) + static_cast<int64_t>(row_ok[m][h] ? row : 0) * n_groups;
      }
    // the scales of a chunk's groups, one chunk ahead of their use
    uint32_t next[MT][2][GPC / 2];
    auto load_scales = [&](int chunk) {
      const int first = chunk * GPC;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const __nv_bfloat16* p = sc[m][h] + first;
          if (a.vec_scales) {
            if constexpr (GPC == 8) {
              const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
              next[m][h][0] = v.x, next[m][h][1] = v.y, next[m][h][2] = v.z, next[m][h][3] = v.w;
            } else if constexpr (GPC == 4) {
              const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
              next[m][h][0] = v.x, next[m][h][1] = v.y;
            } else {
              next[m][h][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
            }
          } else {
#pragma unroll
            for (int j = 0; j < GPC / 2; ++j) {   // groups behind K scale nothing (their activations are zeros)
              const uint32_t lo = first + 2 * j < n_groups ? __bfloat16_as_ushort(p[2 * j]) : 0;
              const uint32_t hi = first + 2 * j + 1 < n_groups ? __bfloat16_as_ushort(p[2 * j + 1]) : 0;
              next[m][h][j] = lo | (hi << 16);
            }
          }
        }
    };
    if (c_lo < c_hi) load_scales(c_lo);
    bool ok = true;
    for (int ch = c_lo; ch < c_hi; ++ch) {
      const int i = ch - c_lo, s = i % NS;
      uint32_t cur[MT][2][GPC / 2];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < GPC / 2; ++j) cur[m][h][j] = next[m][h][j];
      if (ch + 1 < c_hi) load_scales(ch + 1);
      ok = mbar_wait(&sm->full[s], (i / NS) & 1, abort_flag, a.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint8_t* ws = ring + s * C::kStage;
      const uint8_t* xs = ws + C::kWBytes;
      constexpr int JPG = 8 / GPC;     // 32-k steps per group
#pragma unroll
      for (int gr = 0; gr < GPC; ++gr) {
        float part[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) part[m][n][j] = 0.f;
#pragma unroll
        for (int jj = 0; jj < JPG; ++jj) {
          const int j = gr * JPG + jj;         // 16 bytes of codes a row; lane c takes word c: k = 32 j + 8 c ..
          uint32_t fr[MT][2][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = (warp * MT + m) * 16 + g + 8 * h;
              const uint32_t w = *reinterpret_cast<const uint32_t*>(ws + sw128_chunk(r, j) + 4 * c);
#pragma unroll
              for (int q = 0; q < 4; ++q) fr[m][h][q] = w4_pair(w, q);
            }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 x = *reinterpret_cast<const uint4*>(xs + (j >> 1) * C::kXBox +
                                                            sw128_chunk(n * 8 + g, (j & 1) * 4 + c));
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma_16816(part[m][n], fr[m][0][0], fr[m][1][0], fr[m][0][1], fr[m][1][1], x.x, x.y);
              mma_16816(part[m][n], fr[m][0][2], fr[m][1][2], fr[m][0][3], fr[m][1][3], x.z, x.w);
            }
          }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          const uint32_t u0 = cur[m][0][gr >> 1], u1 = cur[m][1][gr >> 1];
          const float s0 = __uint_as_float((gr & 1) ? (u0 & 0xffff0000u) : (u0 << 16));
          const float s1 = __uint_as_float((gr & 1) ? (u1 & 0xffff0000u) : (u1 << 16));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            acc[m][n][0] = fmaf(part[m][n][0], s0, acc[m][n][0]);
            acc[m][n][1] = fmaf(part[m][n][1], s0, acc[m][n][1]);
            acc[m][n][2] = fmaf(part[m][n][2], s1, acc[m][n][2]);
            acc[m][n][3] = fmaf(part[m][n][3], s1, acc[m][n][3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm->empty[s]);
    }
  }
  __syncthreads();
  if (*abort_flag) {   // a wait gave up: let the issued copies land before their memory is used again
    if (warp == kW4Warps && lane == 0)
      for (int i = issued > NS ? issued - NS : 0; i < issued; ++i) mbar_drain(&sm->full[i % NS], (i / NS) & 1);
    __syncthreads();
  }
  griddep_wait();   // y may still be read by an earlier kernel
  // every copy has landed and been read: the ring becomes the partial tile [8 NT tokens][rows]
  float* red = reinterpret_cast<float*>(ring);
  if (warp < kW4Warps) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = (warp * MT + m) * 16 + g + 8 * (j >> 1), t = n * 8 + 2 * c + (j & 1);
          red[t * C::kRows + r] = acc[m][n][j];
        }
  }
  if (splits > 1)
    cluster_sync_all();
  else
    __syncthreads();
  const int tokens = min(8 * NT, a.T - t0);
  const int per = C::kRows / splits;                 // splits is a power of two <= 8
  const int r_lo = rank * per;
  const uint32_t red_addr = smem_u32(red);
  for (int i = threadIdx.x; i < tokens * per; i += kW4Threads) {
    const int t = i / per, r = r_lo + i % per;
    if (row0 + r >= a.N) continue;
    float v = 0.f;
    if (splits > 1) {
      for (int p = 0; p < splits; ++p) v += ld_cluster_f32(cluster_map(red_addr + (t * C::kRows + r) * 4, p));
    } else {
      v = red[t * C::kRows + r];
    }
    static_cast<__nv_bfloat16*>(a.y)[static_cast<int64_t>(t0 + t) * a.N + row0 + r] = __float2bfloat16_rn(v);
  }
  if (splits > 1) cluster_sync_all();   // no CTA leaves while a peer may still read its tile
}

// ---------------------------------------------------------------------------
// many tokens: bf16((code - 8) * scale), 8 codes a thread
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) w4_expand_kernel(W4ExpandArgs a) {
  griddep_wait();   // the workspace may still be read by an earlier product
  griddep_launch_dependents();
  const int k32 = a.K >> 5;
  const int64_t n = static_cast<int64_t>(a.N) * k32;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = i / k32;
    const int k = static_cast<int>(i - row * k32) * 32;
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.codes) + row * (a.K >> 1) + (k >> 1));
    const float s = __bfloat162float(static_cast<const __nv_bfloat16*>(a.scales)[row * (a.K / a.group) + k / a.group]);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + row * a.K + k);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t r[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float v0 = static_cast<float>(static_cast<int>((w[j] >> (8 * q)) & 15u) - 8);
        const float v1 = static_cast<float>(static_cast<int>((w[j] >> (8 * q + 4)) & 15u) - 8);
        r[q] = pack_bf16x2(v0 * s, v1 * s);
      }
      dst[j] = make_uint4(r[0], r[1], r[2], r[3]);
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int NT, int MT, int GPC>
static cudaError_t launch_w4(const W4Args& a, int splits, cudaStream_t st) {
  using C = W4Cfg<NT, MT>;
  auto k = w4_mma_kernel<NT, MT, GPC>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.N + C::kRows - 1) / C::kRows, (a.T + 8 * NT - 1) / (8 * NT), splits);
  prof_begin(st, "w4_mma");
  e = launch_pdl(k, grid, dim3(kW4Threads), C::kSmem, st, splits, a);
  prof_end(st);
  return e;
}

template <int NT, int MT>
static cudaError_t launch_w4_group(const W4Args& a, int splits, cudaStream_t st) {
  switch (a.group) {
    case 32: return launch_w4<NT, MT, 8>(a, splits, st);
    case 64: return launch_w4<NT, MT, 4>(a, splits, st);
    default: return launch_w4<NT, MT, 2>(a, splits, st);
  }
}

W4Plan w4_plan(int N, int T, int K, int num_sms) {
  W4Plan p{};
  p.nt = T <= 8 ? 1 : (T <= 16 ? 2 : (T <= 32 ? 4 : 8));
  // two row tiles a warp share each activation fragment; at 8 token tiles their sums would not fit 168 registers
  p.mt = p.nt == 1 || p.nt == 8 ? 1 : 2;
  p.rows = 16 * p.mt * kW4Warps;
  // K splits: up to 8 (one cluster), while every CTA keeps two chunks and the grid stays near two CTAs an SM
  const int chunks = (K + kW4Chunk - 1) / kW4Chunk;
  const int tiles = ((N + p.rows - 1) / p.rows) * ((T + 8 * p.nt - 1) / (8 * p.nt));
  p.splits = 1;
  while (p.splits < 8 && p.splits * 4 <= chunks && tiles * p.splits * 2 <= 3 * num_sms) p.splits *= 2;
  return p;
}

cudaError_t launch_w4_prep(const W4PrepArgs& a, int num_sms, cudaStream_t st) {
  const int64_t n = static_cast<int64_t>(a.T) * (a.K / 8);
  const int64_t want = (n + 255) / 256;
  const int grid = static_cast<int>(want < 8LL * num_sms ? want : 8LL * num_sms);
  prof_begin(st, "w4_prep");
  cudaError_t e = launch_pdl(w4_prep_kernel, dim3(grid), dim3(256), 0, st, 1, a);
  prof_end(st);
  return e;
}

cudaError_t launch_w4_mma(const W4Args& a, const W4Plan& p, cudaStream_t st) {
  switch (p.nt) {
    case 1: return launch_w4_group<1, 1>(a, p.splits, st);
    case 2: return launch_w4_group<2, 2>(a, p.splits, st);
    case 4: return launch_w4_group<4, 2>(a, p.splits, st);
    default: return launch_w4_group<8, 1>(a, p.splits, st);
  }
}

cudaError_t launch_w4_expand(const W4ExpandArgs& a, int num_sms, cudaStream_t st) {
  const int64_t n = static_cast<int64_t>(a.N) * (a.K / 32);
  const int64_t want = (n + 255) / 256;
  const int grid = static_cast<int>(want < 16LL * num_sms ? want : 16LL * num_sms);
  prof_begin(st, "w4_expand");
  cudaError_t e = launch_pdl(w4_expand_kernel, dim3(grid), dim3(256), 0, st, 1, a);
  prof_end(st);
  return e;
}

}  // namespace gmla
