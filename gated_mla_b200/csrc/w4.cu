// w4.cu — the output product with 4-bit weights and group scales:
//
//   y[t, n] = sum_g scale[n, g] * sum_{k in group g} (code[n, k] - 8) * a[t, k],   a = gate ⊙ o
//
// codes: two per byte (even k in the low nibble), scale: bf16 per row and group of
// 32, 64 or 128 consecutive k.
//
// Few tokens (w4_mma): bound by the weights' N K / 2 bytes, and next to that by
// instruction issue (unpacking a code must cost about one instruction). A row
// tile's codes stream through a ring of TMA boxes (128 rows x 128 bytes = 256 k);
// they become bf16 in registers, straight into the A fragments of m16n8k16
// matrix instructions, and never return to shared memory (tcgen05 would need the
// expanded tile written there: 4 bytes of shared traffic for each byte of codes).
//   * One and-or turns nibbles i and i + 4 of a word into the exact bf16 pair 128 + v,
//     so k and k + 4 sit side by side in the activations too.
//   * sum (v - 8) a = sum (128 + v) a - 136 sum a: the group sums of the activations
//     come from w4_prep, in fp32, and take the place of a subtraction for every pair.
//     (The cancellation costs 136 / 4.6, five bits of fp32's 24. An infinity, or a value near fp32's
//     largest, would cancel to NaN: such a group gives NaN on purpose, and each output that comes out
//     as NaN is taken again from its definition, w4_direct.)
//   * The products of one group are summed in fp32 and only then scaled, so no
//     weight is ever rounded.
// w4_prep applies the gate and stores the activations in the order in which a warp
// reads its B fragments: 512 bytes for each 32 k and 8 tokens, no bank conflict.
// K is split over the CTAs of a cluster, which add their fp32 partial tiles
// through distributed shared memory in a fixed order.
//
// Many tokens (above 256): the codes expand once to fp16 in the workspace (w4_expand), the gated
// activations are stored as fp16 too (w4_wide_prep), and the tcgen05 GEMM of the bf16 path runs on
// them. A code times a scale has 3 + 8 significant bits, fp16's 11, so no weight is rounded (in bf16
// each would be, by 2^-8: at 2000 tokens, 7168 x 8192, an error of 0.0027 instead of 0.0017, nearly
// all of it the result's own rounding). There the operands take 35 + 36 us and the GEMM 228, at 1030 TFLOP/s. What fp16 lacks is range, so each weight row and each token
// row is first multiplied by a power of two that brings its largest element near fp16's top; the
// GEMM's epilogue takes both back. Elements down to 2^-28 of the largest keep their full precision.
#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gmla {

namespace {

constexpr int kW4Warps = 8;               // consumer warps; one more issues the copies
constexpr int kW4Threads = 32 * (kW4Warps + 1);
// One 16-row tile a warp. (Two, which share each activation fragment, with two CTAs an SM instead
// of three, took 21.6 us against 21.8 at 7168 x 16384, one token, but 8.2 against 6.9 at 4096 x 4096.)
constexpr int kW4Rows = 16 * kW4Warps;    // weight rows per CTA
constexpr int kW4WBytes = kW4Rows * 128;  // codes of a stage: 128 bytes (256 k) a row

__device__ __forceinline__ uint32_t w4_pair(uint32_t w, int i) {   // (128 + v_i, 128 + v_{i+4}) as bf16x2
  uint32_t r;
  asm("lop3.b32 %0, %1, 0x000f000f, 0x43004300, 0xea;" : "=r"(r) : "r"(w >> (4 * i)));
  return r;
}

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// `bytes` contiguous bytes (16-byte aligned, a multiple of 16) into shared memory.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// CTAs that share an SM, by their shared memory and registers. (One column tile with two CTAs and a ring of
// five stages: 23.5 us against 23.1 at 7168 x 16384. Two column tiles with three CTAs, three stages each and a
// few spills: 29.4 us against 27.8, and 22.1 against 17.0 at 2048 x 16384.)
constexpr int w4_ctas_per_sm(int nt) { return nt == 1 ? 3 : 2; }

struct W4Smem {
  uint64_t full[4], empty[4];
  int abort;
};

template <int NT>   // token columns in tiles of 8: 1, 2 or 4
struct W4Cfg {
  static constexpr int kXFrag = (kW4Chunk / 32) * NT * 512;    // [8 steps of 32 k][NT][32 lanes][16 bytes]
  static constexpr int kXBytes = kXFrag + 256 * NT;            // then -136 sums [groups of the chunk, up to 8][8 NT] fp32
  static constexpr int kStages = NT == 2 ? 4 : 3;
  // the codes' boxes first (1024-byte aligned for the swizzle), then the activations
  static constexpr int kPitch = kW4Rows + 4;                   // floats between tokens of the partial tile
  static constexpr int kRed = kPitch * 8 * NT * 4;             // fp32 partial tile, over the ring once it has drained
  static constexpr int kRing = kStages * (kW4WBytes + kXBytes) > kRed ? kStages * (kW4WBytes + kXBytes) : kRed;
  static constexpr int kSmem = kRing + 1024 + static_cast<int>(sizeof(W4Smem));
  static constexpr int kCtas = w4_ctas_per_sm(NT);
  static_assert(kStages <= 4, "barriers");
  static_assert(kRing % 8 == 0, "barriers behind the ring");
  static_assert(kCtas * (kSmem + 1024) <= 233472, "shared memory of the CTAs sharing an SM");
};

}  // namespace

// 8 consecutive elements of gate ⊙ o, in fp32
__device__ __forceinline__ void w4_gated8(const W4PrepArgs& a, int t, int k, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.o) + static_cast<int64_t>(t) * a.K + k);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
  if (!a.gate_logits) return;
  if (a.gate_mode == kGateChannel) {
    const float4* z = reinterpret_cast<const float4*>(a.gate_logits + static_cast<int64_t>(t) * a.K + k);
    const float4 z0 = z[0], z1 = z[1];
    const float zz[8] = {z0.x, z0.y, z0.z, z0.w, z1.x, z1.y, z1.z, z1.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= 1.f / (1.f + expf(-zz[j]));
  } else {   // d_h is a multiple of 8: one head for the run
    const float gv = head_gate(a.gate_logits + static_cast<int64_t>(t) * a.H, a.H, k / a.d_h, a.gate_mode, a.gate_topk);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= gv;
  }
}

// Elements from here on (2^100, the bits of a bf16) make their group's sum NaN: below, 128 of them times
// 128 + v stay within 2^115, far from fp32's largest.
constexpr uint32_t kW4Large = 0x7180;

// ---------------------------------------------------------------------------
// a = gate ⊙ o in bf16, in fragment order, and -136 times its sum over each group. (bf16: the
// codes' operand 128 + v is, and both operands of the instruction have one type. So the gated product is rounded
// to 2^-8, as gate_out's is, and the result's error is 0.0023 instead of 0.0017; without a gate nothing is rounded.)
// out: for each token tile of 8 nt and each chunk of 256 k, [8 steps][nt][g * 4 + c][8 bf16]: token 8 n + g of the
// tile, k = 32 step + 8 c + (0 4 1 5 2 6 3 7), then the sums [256 / group][8 nt] fp32 in 256 nt bytes.
// Tokens and k behind the end are zeros. A thread makes one run of 8 k; the runs of a group are
// neighbouring lanes.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256) w4_prep_kernel(W4PrepArgs a) {
  griddep_wait();
  griddep_launch_dependents();   // all earlier kernels are done: the product may begin to load its weights
  const int k8 = a.K256 >> 3;
  const uint32_t n = static_cast<uint32_t>(a.T8) * k8;      // at most 256 tokens, 2^21 runs each
  const int g8 = a.group >> 3;
  for (uint32_t i0 = blockIdx.x * blockDim.x; i0 < n; i0 += gridDim.x * blockDim.x) {   // uniform over a block
    const uint32_t i = i0 + threadIdx.x;
    const int t = static_cast<int>(i / k8);
    const int k = static_cast<int>(i - static_cast<uint32_t>(t) * k8) * 8;
    uint32_t w[4] = {0, 0, 0, 0};
    if (i < n && t < a.T && k < a.K) {
      float v[8];
      w4_gated8(a, t, k, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
    }
    uint4 r;
    r.x = __byte_perm(w[0], w[2], 0x5410);
    r.y = __byte_perm(w[0], w[2], 0x7632);
    r.z = __byte_perm(w[1], w[3], 0x5410);
    r.w = __byte_perm(w[1], w[3], 0x7632);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) sum += __uint_as_float(w[j] << 16) + __uint_as_float(w[j] & 0xffff0000u);
    const uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                                  __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    if ((top & 0xffffu) >= kW4Large || (top >> 16) >= kW4Large) sum = __uint_as_float(0x7fc00000u);
    for (int o = 1; o < g8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (i < n) {
      const int tile = t / (8 * a.nt), tt = t - tile * (8 * a.nt);
      uint8_t* blk = static_cast<uint8_t*>(a.out) +
                     (static_cast<int64_t>(tile) * (a.K256 / kW4Chunk) + k / kW4Chunk) * (a.nt * W4Cfg<1>::kXBytes);
      if (k % a.group == 0)
        reinterpret_cast<float*>(blk + a.nt * W4Cfg<1>::kXFrag)[k % kW4Chunk / a.group * 8 * a.nt + tt] = -136.f * sum;
      reinterpret_cast<uint4*>(blk)[(((k >> 5) & 7) * a.nt + (tt >> 3)) * 32 + (tt & 7) * 4 + ((k >> 3) & 3)] = r;
    }
  }
}

// ---------------------------------------------------------------------------
// y[t, n] from its definition, in 64 bits: for outputs whose sum came out as NaN (large or infinite
// activations; a NaN among the inputs stays one). `x`: the token tile's blocks as w4_prep lays them out,
// tt the token in the tile. One thread an output, over all of K: slow, and rare.
// ---------------------------------------------------------------------------
static __device__ __noinline__ float w4_direct(const W4Args& a, const uint8_t* x, int nt, int tt, int n) {
  const int n_groups = a.K / a.group;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.codes) + static_cast<int64_t>(n) * (a.K >> 1));
  const __nv_bfloat16* scales = static_cast<const __nv_bfloat16*>(a.scales) + static_cast<int64_t>(n) * n_groups;
  double y = 0.0;
  for (int k = 0; k < a.K && y == y; k += 8) {
    const uint8_t* blk = x + static_cast<int64_t>(k / kW4Chunk) * (nt * W4Cfg<1>::kXBytes);
    const uint4 r = reinterpret_cast<const uint4*>(blk)[(((k >> 5) & 7) * nt + (tt >> 3)) * 32 + (tt & 7) * 4 + ((k >> 3) & 3)];
    const uint32_t v[4] = {r.x, r.y, r.z, r.w};      // elements q and q + 4 of the run
    const uint32_t w = codes[k >> 3];
    double sum = 0.0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int lo = static_cast<int>((w >> (4 * q)) & 15u) - 8, hi = static_cast<int>((w >> (4 * q + 16)) & 15u) - 8;
      sum += static_cast<double>(__uint_as_float(v[q] << 16)) * lo;
      sum += static_cast<double>(__uint_as_float(v[q] & 0xffff0000u)) * hi;
    }
    y += sum * static_cast<double>(__bfloat162float(scales[k / a.group]));
  }
  return static_cast<float>(y);
}

// ---------------------------------------------------------------------------
// few tokens, tiles of 8 NT. Grid (row tiles, token tiles, K splits); the splits of a tile form a cluster.
// GPC groups per 256-k chunk (8, 4 or 2).
// ---------------------------------------------------------------------------
template <int NT, int GPC>
__global__ void __launch_bounds__(kW4Threads, W4Cfg<NT>::kCtas) w4_mma_kernel(const __grid_constant__ W4Args a) {
  using C = W4Cfg<NT>;
  constexpr int NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring_x = ring + NS * kW4WBytes;
  W4Smem* sm = reinterpret_cast<W4Smem*>(ring + C::kRing);
  volatile int* abort_flag = &sm->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int splits = gridDim.z, rank = blockIdx.z;
  const int n_chunk = (a.K + kW4Chunk - 1) / kW4Chunk;
  // the splits take the chunks in turn, so that a cluster reads whole stretches of each row at a time
  const int n_c = (n_chunk - rank + splits - 1) / splits;      // chunks rank, rank + splits, ..
  const int row0 = blockIdx.x * kW4Rows;
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

  float acc[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[n][j] = 0.f;

  int issued = 0;   // stages requested (copy thread)
  if (warp == kW4Warps) {
    if (lane == 0) {
      // the weights: w4_prep, the kernel before this one, neither writes them nor starts
      // this one before all earlier kernels are done, so they are requested before the wait
      tma_prefetch_desc(&a.wmap);
      const uint64_t pol_w = l2_evict_first(), pol_x = l2_evict_last();
      const int pre = n_c < NS ? n_c : NS;
      const uint8_t* x = static_cast<const uint8_t*>(a.x) + static_cast<int64_t>(blockIdx.y) * n_chunk * C::kXBytes;
      auto load_w = [&](int i) {
        const int s = i % NS;
        mbar_arrive_expect_tx(&sm->full[s], kW4WBytes + C::kXBytes);
        tma_load_2d(&a.wmap, &sm->full[s], ring + s * kW4WBytes, (rank + i * splits) * 128, row0, pol_w);
      };
      auto load_x = [&](int i) {
        const int s = i % NS;
        bulk_load(ring_x + s * C::kXBytes, x + static_cast<int64_t>(rank + i * splits) * C::kXBytes, C::kXBytes,
                  &sm->full[s], pol_x);
      };
      for (int i = 0; i < pre; ++i) load_w(i);
      griddep_wait();
      for (int i = 0; i < pre; ++i) load_x(i);
      for (issued = pre; issued < n_c; ++issued) {
        if (!mbar_poll<0>(&sm->empty[issued % NS], ((issued / NS) & 1) ^ 1, abort_flag, a.status)) break;
        load_w(issued);
        load_x(issued);
      }
    }
    __syncwarp();
  } else {
    const int g = lane >> 2, c = lane & 3;
    const int n_groups = a.K / a.group;
    const __nv_bfloat16* sc[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = row0 + warp * 16 + g + 8 * h;
      sc[h] = static_cast<const __nv_bfloat16*>(a.scales) + static_cast<int64_t>(row < a.N ? row : 0) * n_groups;
    }
    // the scales of a chunk's groups, one chunk ahead of their use
    uint32_t next[2][GPC / 2];
    auto load_scales = [&](int chunk) {
      const int first = chunk * GPC;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const __nv_bfloat16* p = sc[h] + first;
        if (a.vec_scales) {
          if constexpr (GPC == 8) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
            next[h][0] = v.x, next[h][1] = v.y, next[h][2] = v.z, next[h][3] = v.w;
          } else if constexpr (GPC == 4) {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
            next[h][0] = v.x, next[h][1] = v.y;
          } else {
            next[h][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
          }
        } else {
#pragma unroll
          for (int j = 0; j < GPC / 2; ++j) {   // groups behind K scale nothing (their activations are zeros)
            const uint32_t lo = first + 2 * j < n_groups ? __bfloat16_as_ushort(p[2 * j]) : 0;
            const uint32_t hi = first + 2 * j + 1 < n_groups ? __bfloat16_as_ushort(p[2 * j + 1]) : 0;
            next[h][j] = lo | (hi << 16);
          }
        }
      }
    };
    if (n_c > 0) load_scales(rank);
    // rows g and g + 8 of the warp's 16: word c of the 16-byte chunk j ^ g
    const uint32_t w_off = (warp * 16 + g) * 128 + (g << 4) + 4 * c;
    for (int i = 0; i < n_c; ++i) {
      const int s = i % NS;
      uint32_t cur[2][GPC / 2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < GPC / 2; ++j) cur[h][j] = next[h][j];
      if (i + 1 < n_c) load_scales(rank + (i + 1) * splits);
      bool ok = mbar_poll<20>(&sm->full[s], (i / NS) & 1, abort_flag, a.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint8_t* ws = ring + s * kW4WBytes;
      const uint8_t* xs = ring_x + s * C::kXBytes;
      constexpr int JPG = 8 / GPC;     // 32-k steps per group
#pragma unroll
      for (int gr = 0; gr < GPC; ++gr) {
        float part[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const float2 corr = *reinterpret_cast<const float2*>(xs + C::kXFrag + (gr * 8 * NT + n * 8 + 2 * c) * 4);
          part[n][0] = corr.x, part[n][1] = corr.y, part[n][2] = corr.x, part[n][3] = corr.y;
        }
#pragma unroll
        for (int jj = 0; jj < JPG; ++jj) {
          const int j = gr * JPG + jj;         // 16 bytes of codes a row; lane c takes word c: k = 32 j + 8 c ..
          const uint8_t* wp = ws + (w_off ^ (j << 4));
          const uint32_t w0 = *reinterpret_cast<const uint32_t*>(wp);
          const uint32_t w1 = *reinterpret_cast<const uint32_t*>(wp + 1024);
          uint32_t f0[4], f1[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            f0[q] = w4_pair(w0, q);
            f1[q] = w4_pair(w1, q);
          }
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const uint4 x = *reinterpret_cast<const uint4*>(xs + (j * NT + n) * 512 + lane * 16);
            mma_16816(part[n], f0[0], f1[0], f0[1], f1[1], x.x, x.y);
            mma_16816(part[n], f0[2], f1[2], f0[3], f1[3], x.z, x.w);
          }
        }
        const uint32_t u0 = cur[0][gr >> 1], u1 = cur[1][gr >> 1];
        const float s0 = __uint_as_float((gr & 1) ? (u0 & 0xffff0000u) : (u0 << 16));
        const float s1 = __uint_as_float((gr & 1) ? (u1 & 0xffff0000u) : (u1 << 16));
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[n][0] = fmaf(part[n][0], s0, acc[n][0]);
          acc[n][1] = fmaf(part[n][1], s0, acc[n][1]);
          acc[n][2] = fmaf(part[n][2], s1, acc[n][2]);
          acc[n][3] = fmaf(part[n][3], s1, acc[n][3]);
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
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) red[(n * 8 + 2 * c + (j & 1)) * C::kPitch + warp * 16 + g + 8 * (j >> 1)] = acc[n][j];
  }
  if (splits > 1)
    cluster_sync_all();
  else
    __syncthreads();
  // CTA `rank` adds up its share of the tile's rows, four at a time, over the splits in order
  const int q_lo = (kW4Rows / 4) * rank / splits, q_n = (kW4Rows / 4) * (rank + 1) / splits - q_lo;
  const uint32_t red_addr = smem_u32(red);
  const int t0 = blockIdx.y * 8 * NT, n_t = a.T - t0 < 8 * NT ? a.T - t0 : 8 * NT;
  for (int i = threadIdx.x; i < n_t * q_n; i += kW4Threads) {
    const int t = i / q_n, r = (q_lo + i % q_n) * 4;
    if (row0 + r >= a.N) continue;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (splits > 1) {
      float4 p[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < splits) p[k] = ld_cluster_f32x4(cluster_map(red_addr + (t * C::kPitch + r) * 4, k));
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (k < splits) v.x += p[k].x, v.y += p[k].y, v.z += p[k].z, v.w += p[k].w;
    } else {
      v = *reinterpret_cast<const float4*>(red + t * C::kPitch + r);
    }
    if (!(v.x == v.x && v.y == v.y && v.z == v.z && v.w == v.w)) {
      const uint8_t* x = static_cast<const uint8_t*>(a.x) + static_cast<int64_t>(blockIdx.y) * n_chunk * C::kXBytes;
      float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll 1
      for (int k = 0; k < 4; ++k)
        if (f[k] != f[k] && row0 + r + k < a.N) f[k] = w4_direct(a, x, NT, t, row0 + r + k);
      v = make_float4(f[0], f[1], f[2], f[3]);
    }
    __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + static_cast<int64_t>(t0 + t) * a.N + row0 + r;
    if (a.N % 4 == 0) {
      *reinterpret_cast<uint2*>(y) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    } else {
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (row0 + r + k < a.N) y[k] = __float2bfloat16_rn(f[k]);
    }
  }
  if (splits > 1) cluster_sync_all();   // no CTA leaves while a peer may still read its tile
}

// ---------------------------------------------------------------------------
// Many tokens: one row of fp16 operands a block, and the power of two that its sums are
// multiplied by afterwards. Bound by the bytes that they read and write.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }   // -126 .. 127

// The largest of the block's values (s_top: a word a warp).
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* s_top) {
  v = __reduce_max_sync(0xffffffffu, v);
  if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = v;
  __syncthreads();
  uint32_t top = 0;
  for (int i = 0; i < static_cast<int>(blockDim.x >> 5); ++i) top = max(top, s_top[i]);
  return top;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

constexpr int kWideThreads = 512, kWideVec = 4;   // 16384 k in registers between the maximum and the rounding

__global__ void __launch_bounds__(kWideThreads) w4_wide_prep_kernel(W4PrepArgs a) {
  __shared__ uint32_t s_top[kWideThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x, n8 = a.K >> 3;
  float v[kWideVec][8];
  uint32_t top = 0;      // magnitudes compare as their bits do
#pragma unroll
  for (int i = 0; i < kWideVec; ++i) {
    const int k8 = threadIdx.x + i * kWideThreads;
    if (k8 >= n8) break;
    w4_gated8(a, t, k8 * 8, v[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[i][j]) & 0x7fffffffu);
  }
  for (int k8 = threadIdx.x + kWideVec * kWideThreads; k8 < n8; k8 += kWideThreads) {
    float u[8];
    w4_gated8(a, t, k8 * 8, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(u[j]) & 0x7fffffffu);
  }
  top = block_max(top, s_top);
  const int e = max(-110, min(127, static_cast<int>(top >> 23) - 127));   // 2^e <= largest < 2^(e + 1); infinities and NaN: 127
  const float mul = pow2(14 - e);
  if (threadIdx.x == 0) a.t_scale[t] = pow2(e - 14);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__half*>(a.out) + static_cast<int64_t>(t) * a.K);
  auto store = [&](int k8, const float (&u)[8]) {
    dst[k8] = make_uint4(pack_f16x2(u[0] * mul, u[1] * mul), pack_f16x2(u[2] * mul, u[3] * mul),
                         pack_f16x2(u[4] * mul, u[5] * mul), pack_f16x2(u[6] * mul, u[7] * mul));
  };
#pragma unroll
  for (int i = 0; i < kWideVec; ++i) {
    const int k8 = threadIdx.x + i * kWideThreads;
    if (k8 >= n8) break;
    store(k8, v[i]);
  }
  for (int k8 = threadIdx.x + kWideVec * kWideThreads; k8 < n8; k8 += kWideThreads) {
    float u[8];
    w4_gated8(a, t, k8 * 8, u);
    store(k8, u);
  }
}

__global__ void __launch_bounds__(256) w4_expand_kernel(W4ExpandArgs a) {
  __shared__ uint32_t s_top[8];
  griddep_wait();   // the workspace may still be read by an earlier product
  griddep_launch_dependents();
  const int64_t row = blockIdx.x;
  const int n8 = a.K >> 3, g8 = __ffs(a.group >> 3) - 1, n_groups = a.K / a.group;
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.codes) + row * (a.K >> 1));
  const uint16_t* scales = static_cast<const uint16_t*>(a.scales) + row * n_groups;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<__half*>(a.out) + row * a.K);
  uint32_t top = 0;
  for (int i = threadIdx.x; i < n_groups; i += 256) top = max(top, scales[i] & 0x7fffu);
  top = block_max(top, s_top);
  // the largest scale to 2^11 .. 2^12: 8 of it stay below 2^15
  const int e = max(-100, min(127, static_cast<int>(top >> 7) - 127));
  const float mul = pow2(11 - e);
  if (threadIdx.x == 0) a.f_scale[row] = pow2(e - 11);
#pragma unroll 4
  for (int i = threadIdx.x; i < n8; i += 256) {
    const uint32_t w = codes[i];
    const float s = __uint_as_float(static_cast<uint32_t>(scales[i >> g8]) << 16) * mul;
    float v[8];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t p = w4_pair(w, q);      // 128 + code: exact, and so is the difference
      v[q] = (__uint_as_float(p << 16) - 136.f) * s;
      v[q + 4] = (__uint_as_float(p & 0xffff0000u) - 136.f) * s;
    }
    dst[i] = make_uint4(pack_f16x2(v[0], v[1]), pack_f16x2(v[2], v[3]), pack_f16x2(v[4], v[5]), pack_f16x2(v[6], v[7]));
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
template <int NT, int GPC>
static cudaError_t launch_w4(const W4Args& a, const W4Plan& p, cudaStream_t st) {
  using C = W4Cfg<NT>;
  auto k = w4_mma_kernel<NT, GPC>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid((a.N + kW4Rows - 1) / kW4Rows, p.T8 / (8 * NT), p.splits);
  prof_begin(st, "w4_mma");
  e = launch_pdl(k, grid, dim3(kW4Threads), C::kSmem, st, p.splits, a);
  prof_end(st);
  return e;
}

template <int NT>
static cudaError_t launch_w4_group(const W4Args& a, const W4Plan& p, cudaStream_t st) {
  switch (a.group) {
    case 32: return launch_w4<NT, 8>(a, p, st);
    case 64: return launch_w4<NT, 4>(a, p, st);
    default: return launch_w4<NT, 2>(a, p, st);
  }
}

// Token columns: the smallest of 8, 16 and 32 that holds T, or up to eight tiles of 32, which share a
// row tile's codes in L2. More tokens are left to expansion and GEMM (us at 4096 x 4096 and 7168 x
// 16384: 64 tokens 16.7 and 73, 128 tokens 24 and 136, 256 tokens 39 and 240; expansion and GEMM take 62
// and 267 from 257 to 512 tokens). K splits: the number (1 .. 8, one cluster) with the least time,
// counted as waves of resident clusters times the chunks that each CTA works through plus about two
// chunks' time for its start and its sum. A cluster stays within one of the 8 GPCs, and w4_prep's last CTAs
// still hold slots when it is placed: a sixteenth of what fits is left out. (One token at 7168 x 16384: 56
// clusters of 7, just what fits, took 22 us in a stream but two waves and 36 us in a graph; of 6 they take 23
// and 25. 16 tokens at 4096 x 4096: 32 of 8 13.5 us, of 6 9.6. 32 tokens at 7168 x 16384: 56 of 5 51 us, of 4 41.)
W4Plan w4_plan(int N, int T, int K, int num_sms) {
  W4Plan p{};
  p.T8 = T;
  p.K256 = K;
  if (T > kW4MaxMma) return p;
  const int chunks = (K + kW4Chunk - 1) / kW4Chunk;
  p.nt = T <= 8 ? 1 : (T <= 16 ? 2 : 4);
  const int token_tiles = (T + 8 * p.nt - 1) / (8 * p.nt);
  const int64_t tiles = static_cast<int64_t>((N + kW4Rows - 1) / kW4Rows) * token_tiles;
  int64_t best = 0;
  for (int s = 1; s <= 8 && s <= chunks; ++s) {
    const int64_t fit = 8 * (num_sms / 8 * w4_ctas_per_sm(p.nt) / s), room = fit > 16 ? fit - fit / 16 : 1;
    const int64_t cost = ((tiles + room - 1) / room) * ((chunks + s - 1) / s + 2);
    if (s == 1 || cost < best) best = cost, p.splits = s;
  }
  p.T8 = 8 * p.nt * token_tiles;
  p.K256 = chunks * kW4Chunk;
  return p;
}

cudaError_t launch_w4_prep(const W4PrepArgs& a, int num_sms, cudaStream_t st) {
  const int64_t n = static_cast<int64_t>(a.T8) * (a.K256 / 8);
  const int64_t want = (n + 255) / 256;
  const int grid = static_cast<int>(want < 8LL * num_sms ? want : 8LL * num_sms);
  prof_begin(st, "w4_prep");
  cudaError_t e = launch_pdl(w4_prep_kernel, dim3(grid), dim3(256), 0, st, 1, a);
  prof_end(st);
  return e;
}

cudaError_t launch_w4_wide_prep(const W4PrepArgs& a, cudaStream_t st) {
  prof_begin(st, "w4_wide_prep");
  cudaError_t e = launch_pdl(w4_wide_prep_kernel, dim3(a.T), dim3(kWideThreads), 0, st, 1, a);
  prof_end(st);
  return e;
}

cudaError_t launch_w4_mma(const W4Args& a, const W4Plan& p, cudaStream_t st) {
  switch (p.nt) {
    case 1: return launch_w4_group<1>(a, p, st);
    case 2: return launch_w4_group<2>(a, p, st);
    default: return launch_w4_group<4>(a, p, st);
  }
}

cudaError_t launch_w4_expand(const W4ExpandArgs& a, cudaStream_t st) {
  prof_begin(st, "w4_expand");
  cudaError_t e = launch_pdl(w4_expand_kernel, dim3(a.N), dim3(256), 0, st, 1, a);
  prof_end(st);
  return e;
}

}  // namespace gmla
