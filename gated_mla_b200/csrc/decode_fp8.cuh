// decode_fp8.cuh — absorbed-form decode over an FP8 (E4M3) latent cache
// (included at the end of decode_tc.cu: it shares the split plan and the merge).
//
// The cache holds e4m3 codes c~ with one fp32 scale for the whole cache
// (c = cache_scale * c~), half the bytes of a bf16 cache. The method is that of
// decode_tc.cu ("Gated MLA 计算公式" §一/§二, "精读笔记 03" §5.1, 题4):
//   z_s = q_lat . c_s,  O_lat = sum_s softmax(z)_s c_s,  o = W_v O_lat (gated).
// Both products run on tcgen05 kind::f8f6f4 tensor cores straight from the
// cached codes (no conversion pass):
//   S^T = C~ (Q~)^T   M = 128 tokens, K = 32 latent dims per MMA, N = 2 HG
//   O^T += C~^T P^T   M = 128 latent dims (the cache box read MN-major), K = 32 tokens
// The other operand of each product is not an FP8 quantity of the method, so it
// is carried as a hi + lo pair of e4m3 values (v ~ hi + lo, about 7 significant
// bits): the absorbed query as Q~ = [hi(q_lat / sigma); lo(...)] with one scale
// sigma per (sequence, head), and P' = kPScale p as [hi; lo]. The pair doubles N,
// which costs next to nothing at these widths (an MMA with N <= 64 is bound by
// its A operand). Scores are (S[h] + S[HG + h]) * sigma * cache_scale; the
// weighted sum is (O^T[h] + O^T[HG + h]) * cache_scale / kPScale.
//
// With one scale s_t for every block of token rows (BLK; c = s_t c~) the weighted
// sum's weights are p_t s_t, whose spread adds to that of p_t. So the running
// reference m follows u_t = z_t + log2 s_t, P' = kPScaleB 2^(u - m) carries the scale
// into the product, and the softmax sum takes 2^(u - m) / s_t. P' gets a third
// e4m3 term, and each term is stored 32 times finer than the one before
// (P' = hi + lo / 32 + lo2 / 1024, in columns of their own), a grid of 2^-22 of the
// reference. Rounding to the nearest would drop every weight below 2^-23, and with
// them the whole tail of a long context that one token far outweighs (131071 rows at
// 2^-23 are 1.6 % of the softmax), though the denominator counts it. So the last term is
// rounded with an offset of each token's own, spread evenly over a step: a weight w is
// stored as 0 or 2^-22 (the two grid points around it) in the ratio that makes a sum over
// many tokens come out right (to a few steps in all), however small w is. At N = 3 HG <= 96 an
// MMA costs what it does at 2 HG.
//
// Kernels: decode_absorb_fp8, with block scales decode_absorb_tc8 (q_lat, its scale and
// hi/lo codes; its last block builds the split plan as decode_absorb_plan does),
// decode_attn_fp8 (below), then decode_merge and the W_v GEMM of the bf16 path.
//
// Block scales, attention alone: 64 paged sequences, 32 heads 85 us, where reading the codes takes
// 35; 8 sequences of 131072 rows, 128 heads 485 us, of which the MMAs of the three-term product
// and the tile's softmax take turns (the codes take 88).
#pragma once
#include <cuda_fp8.h>

namespace gmla {

namespace {
constexpr int kTok = 128;                  // tokens per tile
constexpr int kBox8 = 128 * 128;           // one box: 128 token rows x 128 e4m3 latent dims
constexpr int kNB8 = 4;                    // boxes per tile (d_c = 512)
constexpr int kDc8 = 512;
// The running max of a head is raised only when a tile's max exceeds it by
// more than kRaise8 (log2 units), so p = 2^(s - m) <= 2^kRaise8 and
// P' = kPScale p <= 256, inside E4M3's range (448); weights down to
// 2^-15 stay representable.
constexpr float kRaise8 = 2.f;
constexpr float kPScale = 64.f;
// With three terms (block scales) the same P' <= 256 leaves room for a raise only every 5 log2
// units (a raise rescales O in tensor memory, nearly a tile's time), on a grid of
// 2^-22 of the reference.
constexpr float kRaise8B = 5.f;
constexpr float kPScaleB = 8.f;

__device__ __forceinline__ uint8_t to_e4m3(float v) {
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3));
}
__device__ __forceinline__ float from_e4m3(uint8_t c) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(c), __NV_E4M3);
  return __half2float(__half(h));
}
// hi + lo e4m3 pair of v (hi = e4m3(v), lo = e4m3(v - hi))
__device__ __forceinline__ void split_e4m3(float v, uint8_t& hi, uint8_t& lo) {
  hi = to_e4m3(v);
  lo = to_e4m3(v - from_e4m3(hi));
}
// The rounding offset of a token's last term: up to half of E4M3's smallest step (2^-9) either way. Multiples of the
// golden ratio, modulo 1, by position: any stretch of tokens has them nearly even.
__device__ __forceinline__ float term_offset(int pos) {
  return static_cast<float>(static_cast<int>(static_cast<uint32_t>(pos) * 2654435769u)) * 4.547473508864641e-13f;   // 2^-41
}
// Two values as e4m3 terms, `n` of them, each 32 times finer than the one before
// (v = t0 + t1 / 32 + t2 / 1024): codes of the pair in the low two bytes of t[i]. `offset` goes to the
// last term before it is rounded (0 stays 0).
template <int n>
__device__ __forceinline__ void terms_e4m3x2(float a, float b, float offset, uint32_t (&t)[n]) {
#pragma unroll
  for (int i = 0; i < n; ++i) {
    const __nv_fp8x2_storage_t c = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    t[i] = c;
    if (i + 1 < n) {
      const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(c, __NV_E4M3));
      const float d = i + 2 == n ? offset : 0.f;
      a = fmaf(a - __low2float(h), 32.f, d);
      b = fmaf(b - __high2float(h), 32.f, d);
    }
  }
}
// byte offset of (row, col) in a K-major tile of 128-byte rows with the 128-byte swizzle
__device__ __forceinline__ uint32_t sw128_byte(uint32_t row, uint32_t col) {
  return row * 128u + ((((col >> 4) ^ row) & 7u) << 4) + (col & 15u);
}
}  // namespace

// ---------------------------------------------------------------------------
// absorb: per (head, 8 sequences): q_lat = q_scale * W_k^(h)T q^(h) over all 512
// latent dims, sigma = max |q_lat| / 448, codes hi/lo of q_lat / sigma written to
// the rows of the head's slot; qmul = sigma * cache_scale. The last block runs
// the split plan.
// ---------------------------------------------------------------------------
constexpr int kAbs8B = 8;

__global__ void __launch_bounds__(256) decode_absorb_fp8_kernel(DecodeArgs a) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  const int n_bblk = (a.B + kAbs8B - 1) / kAbs8B;
  if (static_cast<int>(blockIdx.x) == a.H * n_bblk) {
    griddep_wait();
    decode_plan_block(a);
    return;
  }
  const int h = blockIdx.x / n_bblk;
  const int b0 = (blockIdx.x % n_bblk) * kAbs8B;
  const int nb = min(kAbs8B, a.B - b0);
  const int c0 = threadIdx.x * 2;   // two latent columns per thread
  const __nv_bfloat16* Wk = static_cast<const __nv_bfloat16*>(a.W_k) + static_cast<int64_t>(h) * a.d_h * kDc8;
  __shared__ float sq[kAbs8B][256];
  __shared__ float red[kAbs8B][8];
  __shared__ int s_slot[kAbs8B];
  __shared__ float s_on[kAbs8B];
  griddep_wait();
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q);
  const int dq = a.d_h + a.d_rope;
  for (int i = threadIdx.x; i < kAbs8B * a.d_h; i += blockDim.x) {
    const int bi = i / a.d_h, k = i % a.d_h;
    sq[bi][k] = bi < nb ? __bfloat162float(q[(static_cast<int64_t>(b0 + bi) * a.H + h) * dq + k]) : 0.f;
  }
  if (threadIdx.x < kAbs8B) {
    int slot = h;
    float on = 1.f;
    const int bi = threadIdx.x;
    if (a.gate_hard && bi < nb) {
      const float* z = a.gate_logits + static_cast<int64_t>(b0 + bi) * a.H;
      int na = 0;
      slot = head_slot(z, a.H, h, a.gate_mode, a.gate_topk, &na);
      const float gv = head_gate(z, a.H, h, a.gate_mode, a.gate_topk);
      on = gv != 0.f ? 1.f : 0.f;
      a.gvals[static_cast<int64_t>(b0 + bi) * a.H + h] = gv;
      a.head_of_slot[static_cast<int64_t>(b0 + bi) * a.H + slot] = h;
    }
    s_slot[bi] = slot;
    s_on[bi] = on;
  }
  __syncthreads();
  float acc[kAbs8B][2];
#pragma unroll
  for (int bi = 0; bi < kAbs8B; ++bi) acc[bi][0] = acc[bi][1] = 0.f;
  // 16 rows of W_k in flight at a time (the loads, not the FMAs, set the pace)
  constexpr int kRows = 16;
  for (int k0 = 0; k0 < a.d_h; k0 += kRows) {
    __nv_bfloat162 w2[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      w2[i] = k0 + i < a.d_h ? *reinterpret_cast<const __nv_bfloat162*>(Wk + static_cast<int64_t>(k0 + i) * kDc8 + c0)
                             : __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (k0 + i >= a.d_h) break;
      const float w0 = __low2float(w2[i]), w1 = __high2float(w2[i]);
#pragma unroll
      for (int bi = 0; bi < kAbs8B; ++bi) {
        acc[bi][0] = fmaf(sq[bi][k0 + i], w0, acc[bi][0]);
        acc[bi][1] = fmaf(sq[bi][k0 + i], w1, acc[bi][1]);
      }
    }
  }
  // per sequence: the largest |q_lat| over the 512 dims (block reduction)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int bi = 0; bi < kAbs8B; ++bi) {
    acc[bi][0] *= a.q_scale;
    acc[bi][1] *= a.q_scale;
    float mx = fmaxf(fabsf(acc[bi][0]), fabsf(acc[bi][1]));
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    if (lane == 0) red[bi][warp] = mx;
  }
  __syncthreads();
  uint8_t* qa = static_cast<uint8_t*>(a.qa);
  const int N2 = 2 * a.HG;
  for (int bi = 0; bi < nb; ++bi) {
    float mx = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) mx = fmaxf(mx, red[bi][w]);
    const float sigma = mx > 0.f ? mx / 448.f : 1.f;
    const float inv = 1.f / sigma;
    const int b = b0 + bi, slot = s_slot[bi];
    if (threadIdx.x == 0) a.qmul[static_cast<int64_t>(b) * a.H + slot] = sigma * a.cache_scale * s_on[bi];
    // slots past the launched head groups (heads a top-k gate switches off) are never read
    if (slot >= a.n_hg * a.HG) continue;
    const int64_t row_hi = (static_cast<int64_t>(b) * a.n_hg + slot / a.HG) * N2 + slot % a.HG;
    uint8_t h0, l0, h1, l1;
    split_e4m3(acc[bi][0] * inv * s_on[bi], h0, l0);
    split_e4m3(acc[bi][1] * inv * s_on[bi], h1, l1);
    *reinterpret_cast<uint16_t*>(qa + row_hi * kDc8 + c0) = static_cast<uint16_t>(h0 | (h1 << 8));
    *reinterpret_cast<uint16_t*>(qa + (row_hi + a.HG) * kDc8 + c0) = static_cast<uint16_t>(l0 | (l1 << 8));
  }
}

// ---------------------------------------------------------------------------
// The same for a block-scaled cache, on tcgen05: one CTA per (head, 128 latent columns,
// up to 128 sequences) as decode_absorb_tc; the four column CTAs of a head form a
// cluster and exchange each sequence's largest |q_lat| through distributed shared
// memory, since the codes of all 512 columns share one sigma. Latency bound (64
// sequences, 32 heads: 20 us on CUDA cores, which read W_k once for 8 sequences).
// Grid (heads + 1, sequence chunks, 4); the last x runs the split plan.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(128) decode_absorb_tc8_kernel(const __grid_constant__ DecodeArgs a) {
  if (threadIdx.x == 0) griddep_launch_dependents();
  if (static_cast<int>(blockIdx.x) == a.H) {   // whole clusters
    if (blockIdx.y == 0 && blockIdx.z == 0) {
      griddep_wait();
      decode_plan_block(a);
    }
    return;
  }
  extern __shared__ uint8_t smem_raw[];
  __shared__ float s_wmax[4][128], s_max[128];
  __shared__ float2 s_row[128];   // 1 / sigma (scaled), and the row of a sequence's hi codes (-1: none)
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int BN = a.absorb_bn;
  const int nkb = a.d_h / 64;
  uint8_t* sA = smem;                                  // 2 boxes [d_h rows][64 latent columns]
  uint8_t* sB = sA + 2 * a.d_h * 128;                  // nkb boxes [BN sequences][64 of d_h]
  AbsorbSmem* sm = reinterpret_cast<AbsorbSmem*>(sB + nkb * BN * 128);
  volatile int* abort_flag = &sm->abort;
  const int h = blockIdx.x, ct = blockIdx.z;
  const int b0 = blockIdx.y * BN;
  const int nb = min(BN, a.B - b0);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tcols = BN <= 32 ? 32 : (BN <= 64 ? 64 : 128);
  if (threadIdx.x == 0) {
    mbar_init(&sm->full, 1);
    mbar_init(&sm->mma_done, 1);
    sm->abort = 0;
    fence_mbar_init();
  }
  if (warp == 0) {
    tmem_alloc(&sm->tmem, tcols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm->tmem;
  bool mma_issued = false;   // thread 0
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&a.wk_map);
    tma_prefetch_desc(&a.q_map);
    mbar_arrive_expect_tx(&sm->full, 2u * a.d_h * 128 + static_cast<uint32_t>(nkb * BN * 128));
    for (int j = 0; j < 2; ++j)
      tma_load_2d(&a.wk_map, &sm->full, sA + j * a.d_h * 128, ct * kAbsorbM + j * 64, h * a.d_h, l2_evict_first());
  }
  griddep_wait();   // the queries come from the kernel before this one
  if (threadIdx.x == 0)
    for (int kb = 0; kb < nkb; ++kb)
      tma_load_2d(&a.q_map, &sm->full, sB + kb * BN * 128, h * a.d_h + kb * 64, b0, l2_evict_last());
  if (threadIdx.x < nb) {   // hard / quantised gates: heads by slot, as decode_absorb_tc
    int slot = h;
    float on = 1.f;
    if (a.gate_hard) {
      const int b = b0 + threadIdx.x;
      const float* z = a.gate_logits + static_cast<int64_t>(b) * a.H;
      int na = 0;
      slot = head_slot(z, a.H, h, a.gate_mode, a.gate_topk, &na);
      const float gv = head_gate(z, a.H, h, a.gate_mode, a.gate_topk);
      on = gv != 0.f ? 1.f : 0.f;
      if (ct == 0) {
        a.gvals[static_cast<int64_t>(b) * a.H + h] = gv;
        a.head_of_slot[static_cast<int64_t>(b) * a.H + slot] = h;
      }
    }
    sm->slot[threadIdx.x] = slot;
    sm->on[threadIdx.x] = on;
  }
  if (threadIdx.x == 0) {
    if (mbar_poll<0>(&sm->full, 0, abort_flag, a.status)) {
      tc_fence_after();
      const uint32_t idesc = idesc_bf16_f32(128, BN, true, false);
      const uint64_t dA = sdesc_sw128(smem_u32(sA), a.d_h * 128, 1024);
      const uint64_t dB = sdesc_sw128(smem_u32(sB), 16, 1024);
      for (int k = 0; k < a.d_h / 16; ++k)
        umma_bf16(tmem, dA + (k * 2048) / 16, dB + ((k >> 2) * BN * 128 + (k & 3) * 32) / 16, idesc, k != 0);
      umma_commit(&sm->mma_done);
      mma_issued = true;
    } else {
      mbar_drain(&sm->full, 0);   // copies still in flight land before the block leaves
    }
  }
  __syncthreads();
  bool ok = !*abort_flag && mbar_poll<0>(&sm->mma_done, 0, abort_flag, a.status);
  ok = __all_sync(0xffffffffu, ok);
  // warp w holds latent columns ct*128 + 32 w + lane, one TMEM column per sequence
  const uint32_t taddr = tmem + (static_cast<uint32_t>(32 * warp) << 16);
  if (ok) {
    tc_fence_after();
    for (int n0 = 0; n0 < BN; n0 += 16) {
      uint32_t v[16];
      tmem_ld16(taddr + n0, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) {   // magnitudes order as their bits do
        const uint32_t top = __reduce_max_sync(0xffffffffu, v[j] & 0x7fffffffu);
        if (lane == 0) s_wmax[warp][n0 + j] = __uint_as_float(top);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < BN) {
    const int n = threadIdx.x;
    s_max[n] = ok ? fmaxf(fmaxf(s_wmax[0][n], s_wmax[1][n]), fmaxf(s_wmax[2][n], s_wmax[3][n])) : 0.f;
  }
  cluster_sync_all();
  if (threadIdx.x < BN) {
    const int n = threadIdx.x;
    float mx = 0.f;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_map(smem_u32(&s_max[n]), r)) : "memory");
      mx = fmaxf(mx, v);
    }
    const float sigma = mx > 0.f ? mx * a.q_scale / 448.f : 1.f;
    int row = -1;
    if (n < nb) {   // slots past the launched head groups (heads a top-k gate switches off) are never read
      const int slot = sm->slot[n];
      if (slot < a.n_hg * a.HG) row = ((b0 + n) * a.n_hg + slot / a.HG) * 2 * a.HG + slot % a.HG;
    }
    s_row[n] = make_float2(n < nb ? a.q_scale / sigma * sm->on[n] : 0.f, __int_as_float(row));
    if (ct == 0 && n < nb) a.qmul[static_cast<int64_t>(b0 + n) * a.H + sm->slot[n]] = sigma * a.cache_scale * sm->on[n];
  }
  cluster_sync_all();   // every peer has read the maxima; s_row is written
  if (ok) {
    uint8_t* qa = static_cast<uint8_t*>(a.qa) + ct * kAbsorbM + 32 * warp + lane;
    const int lo_off = a.HG * kDc8;
    for (int n0 = 0; n0 < nb; n0 += 16) {
      uint32_t v[16];
      tmem_ld16(taddr + n0, v);
      tmem_ld_wait();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float2 r = s_row[n0 + j];
        const int row = __float_as_int(r.y);
        if (row < 0) continue;
        uint8_t hi, lo;
        split_e4m3(__uint_as_float(v[j]) * r.x, hi, lo);
        uint8_t* dst = qa + static_cast<int64_t>(row) * kDc8;
        dst[0] = hi;
        dst[lo_off] = lo;
      }
    }
  } else if (mma_issued) {
    mbar_drain(&sm->mma_done, 0);   // an issued product completes before TMEM is freed
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, tcols);
  }
}

// ---------------------------------------------------------------------------
// attention over the FP8 cache
// ---------------------------------------------------------------------------
struct Dec8Smem {
  uint64_t full[16], empty[16];   // per ring box
  uint64_t s_full[2], p_full[2], pv_done[2];   // of even and odd tiles where two tiles are in work (kPipe), else the first
  uint64_t q_full, q_empty, o_done, o_free, drain, never;
  uint32_t tmem;
  int abort;
  int vote[3];
  int red[2][4][64];
  float lred[4][64];
  float mfin[64];
};

// 16 heads per CTA: two CTAs share an SM (each holds a ring of 5 boxes, and
// the 256 columns of tensor memory it needs), so one CTA's loads, softmax and
// MMAs overlap the other's; each CTA on its own is bound by the latency of
// that chain, not by bandwidth. 32 heads: one CTA per SM with a deeper ring.
// Waits of the producer and the softmax warps.
template <bool BLK>
__device__ __forceinline__ bool wait8(uint64_t* bar, uint32_t parity, volatile int* abort, int* status) {
  return BLK ? mbar_poll<20>(bar, parity, abort, status) : mbar_wait(bar, parity, abort, status);
}

template <int HG, bool BLK>
struct Dec8Cfg {
  static constexpr int kN2 = 2 * HG;                         // hi and lo columns of the scores
  static constexpr int kTerms = BLK ? 3 : 2;                 // e4m3 terms of P'
  static constexpr int kNP = kTerms * HG;                    // columns of P' and of O^T
  static constexpr int kSG = HG >= 32 ? 2 : 1;               // softmax warp groups (head slices)
  static constexpr int kThreads = 64 + 128 * kSG + (BLK && HG == 32 ? 32 : 0);
  static constexpr int kCtasPerSm = HG == 16 ? 2 : 1;
  static constexpr int kQBytes = kNB8 * kN2 * 128;           // 4 boxes of [2 HG rows x 128 B]
  // Where the ring holds two tiles (32 heads, block scales) there are two P buffers and two
  // issuing warps, one for the scores and one for the weighted sums: the scores of a tile
  // are complete, and its softmax runs, while the weighted sum of the tile before is still
  // being taken. The ring's boxes go in pairs, a barrier each: even a wait for something
  // complete costs its warp about 250 cycles. (8 x 131072 tokens, 128 heads: in turn 575 us,
  // two P buffers and one issuing warp 557.)
  static constexpr bool kPipe = BLK && HG == 32;
  static constexpr int kPBuf = ((kNP * 128) + 1023) & ~1023;     // [terms x HG rows x 128 tokens]
  static constexpr int kPBytes = (kPipe ? 2 : 1) * kPBuf;
  static constexpr int kStruct = (static_cast<int>(sizeof(Dec8Smem)) + 127) & ~127;
  static constexpr int kFixed = kQBytes + kPBytes + kStruct + 1024 /*align*/;
  // shared memory of an SM (233472 B) less 1 KB reserved per CTA
  static constexpr int kBudget = kCtasPerSm == 2 ? 233472 / 2 - 1024 : 232448;
  static constexpr int kRingMax = (kBudget - kFixed) / kBox8;
  static constexpr int kPair = kPipe ? 2 : 1;                // boxes a barrier
  static constexpr int kRing = (kRingMax > 16 ? 16 : kRingMax) / kPair * kPair;
  static constexpr int kSmem = kRing * kBox8 + kFixed;
  static constexpr int kTmemCols = 2 * kN2 + 4 * kNP <= 256 ? 256 : 512;   // 2 S^T buffers + 4 O^T chunks
  // the next tile's boxes are probed by the parity of their full barrier, which
  // is unambiguous while box c - kRing has been waited for: true up to c =
  // (first box of this tile) + 2 kNB8 - 1 when kRing >= kNB8
  static_assert(kRing >= (kPipe ? 2 * kNB8 : kNB8 + 1), "the ring holds more than one tile, or two");
  static_assert(2 * kN2 + 4 * kNP <= kTmemCols, "scores and sums fit tensor memory");
  static_assert(kCtasPerSm * kTmemCols <= 512, "tensor memory of the CTAs sharing an SM");
};

template <int HG, bool BLK>
__global__ void __launch_bounds__(64 + 128 * (HG >= 32 ? 2 : 1) + (BLK && HG == 32 ? 32 : 0), (HG == 16 ? 2 : 1))
    decode_attn_fp8_kernel(const __grid_constant__ DecodeArgs a) {
  using C = Dec8Cfg<HG, BLK>;
  constexpr int NR = C::kRing, N2 = C::kN2, NP = C::kNP, BP = C::kPair;
  constexpr int NB = NR / BP;      // barriers of the ring: box c has number c / BP
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ring = smem;
  uint8_t* qs = ring + NR * kBox8;
  uint8_t* pbuf = qs + C::kQBytes;
  Dec8Smem* sm = reinterpret_cast<Dec8Smem*>(pbuf + C::kPBytes);
  volatile int* abort_flag = &sm->abort;

  const int g = blockIdx.x, hg = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int heads_valid = min(HG, a.H - hg * HG);
  if (threadIdx.x == 0) {
    for (int i = 0; i < NR; ++i) {
      mbar_init(&sm->full[i], 1);
      mbar_init(&sm->empty[i], 1);
    }
    mbar_init(&sm->q_full, 1);
    mbar_init(&sm->q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->s_full[i], 1);
      mbar_init(&sm->p_full[i], 128 * C::kSG);
      mbar_init(&sm->pv_done[i], 1);
    }
    mbar_init(&sm->o_done, 1);
    mbar_init(&sm->o_free, 128 * C::kSG);
    mbar_init(&sm->drain, C::kPipe ? 2 : 1);
    mbar_init(&sm->never, 1);
    sm->abort = 0;
    sm->vote[0] = sm->vote[1] = sm->vote[2] = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm->tmem, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) griddep_launch_dependents();
  griddep_wait();   // the plan, the absorbed queries and the cache rows come from earlier kernels
  const int seg_lo = a.cta_first_seg[g];
  const int seg_hi = (seg_lo < a.cta_first_seg[g + 1]) ? a.cta_first_seg[g + 1] : seg_lo;
  const uint32_t tmem = sm->tmem;
  const uint32_t tO = tmem + 2 * N2;   // O^T chunk j (latent dims 128 j ..) at columns tO + j NP
  uint32_t loaded = 0, loaded_q = 0;   // ring boxes and query tiles requested (producer)

  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    if (lane == 0) {
      tma_prefetch_desc(&a.cache_map);
      tma_prefetch_desc(&a.qa_map);
    }
    const uint64_t pol_c = a.n_hg > 1 ? l2_evict_normal() : l2_evict_first();
    const uint64_t pol_q = l2_evict_last();
    const bool paged = a.cache.paged != 0;
    const int ps = paged ? a.cache.page_size : kTok;
    uint32_t nbox = 0, nq = 0;
    bool ok = true;
    for (int si = seg_lo; si < seg_hi && ok; ++si) {
      const int4 sg = a.seg_info[si];
      const int b = sg.x;
      const int L = sg.w;
      if (seg_heads(a, b, hg, heads_valid) == 0) continue;
      if (lane == 0) {
        if (nq > 0 && !wait8<BLK>(&sm->q_empty, (nq - 1) & 1, abort_flag, a.status)) ok = false;
        if (ok) {
          mbar_arrive_expect_tx(&sm->q_full, C::kQBytes);
          for (int j = 0; j < kNB8; ++j)
            tma_load_2d(&a.qa_map, &sm->q_full, qs + j * N2 * 128, j * 128, (b * a.n_hg + hg) * N2, pol_q);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      ++nq;
      for (int t = sg.y; t < sg.z && ok; ++t) {
        const int tok0 = t * kTok;
        const int valid = min(kTok, L - tok0);
        const int nchunk = ps >= kTok ? 1 : (valid + ps - 1) / ps;   // <= 16 (page size >= 8)
        int page = 0;
        if (paged && lane < nchunk)
          page = a.cache.block_table[static_cast<int64_t>(b) * a.cache.max_pages_per_seq + (tok0 + lane * ps) / ps];
        const uint32_t tx = ps >= kTok ? kBox8 : nchunk * ps * 128;
        for (int j = 0; j < kNB8; ++j) {
          const uint32_t slot = nbox % NR, nb = nbox / BP, bs = nb % NB;
          if (j % BP == 0) {
            if (lane == 0) {
              if (nb >= static_cast<uint32_t>(NB) &&
                  !wait8<BLK>(&sm->empty[bs], ((nb / NB) & 1) ^ 1, abort_flag, a.status))
                ok = false;
              if (ok) mbar_arrive_expect_tx(&sm->full[bs], BP * tx);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
          }
          uint8_t* dst = ring + slot * kBox8;
          if (!paged) {
            if (lane == 0) tma_load_2d(&a.cache_map, &sm->full[bs], dst, j * 128, b * a.cache.capacity + tok0, pol_c);
          } else if (ps >= kTok) {
            if (lane == 0) tma_load_3d(&a.cache_map, &sm->full[bs], dst, j * 128, tok0 % ps, page, pol_c);
          } else if (lane < nchunk) {
            tma_load_3d(&a.cache_map, &sm->full[bs], dst + lane * ps * 128, j * 128, 0, page, pol_c);
          }
          ++nbox;
        }
      }
    }
    loaded = nbox;
    loaded_q = nq;
  } else if (warp == 1 || (C::kPipe && warp == C::kThreads / 32 - 1)) {
    // ------------------------------ MMA issuers ------------------------------
    if constexpr (BLK) {   // whole warps, converged (see umma_f8_warp)
      constexpr uint32_t idS = idesc_e4m3_f32(128, N2, false, false);
      constexpr uint32_t idO = idesc_e4m3_f32(128, NP, true, false);
      const uint32_t ring_a = smem_u32(ring);
      const uint64_t dRing = sdesc_sw128(ring_a, 16, 1024), dQ = sdesc_sw128(smem_u32(qs), 16, 1024);
      const uint64_t dRingMN = sdesc_sw128(ring_a, kBox8, 1024);   // a box read as [tokens (K) x 128 latent dims (M)]
      const uint64_t dP = sdesc_sw128(smem_u32(pbuf), 16, 1024);
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_poll<0>(bar, parity, abort_flag, a.status)) != 0;
      };
      auto s_box = [&](uint32_t slot, int j, uint32_t tSb) {   // S^T += box j of the tile x its Q box
        const uint64_t da = dRing + slot * (kBox8 / 16);
        const uint64_t db = dQ + j * (N2 * 128 / 16);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma_f8_warp(tSb, da + kk * 2, db + kk * 2, idS, (j | kk) != 0);
      };
      uint32_t nbox = 0, ntile = 0, nseg = 0;
      bool ok = true;
      // scores of the tile at nbox, its boxes from `from` on, into buffer ntile & 1
      auto scores = [&](int from) {
        for (int j = from; j < kNB8 && ok; ++j) {
          const uint32_t nb = (nbox + j) / BP;
          if (j % BP == 0) ok = wait(&sm->full[nb % NB], (nb / NB) & 1);
          if (ok) s_box((nbox + j) % NR, j, tmem + (ntile & 1) * N2);
        }
      };
      // O^T += C~^T P'^T of the tile at nbox; its boxes are free when this is done
      auto weighted_sum = [&](bool first) {
        tc_fence_after();
        const uint64_t dPb = dP + (C::kPipe ? (ntile & 1) * (C::kPBuf / 16) : 0);
#pragma unroll 1
        for (int j = 0; j < kNB8; ++j) {
          const uint64_t da = dRingMN + (nbox + j) % NR * (kBox8 / 16);
#pragma unroll
          for (int kk = 0; kk < kTok / 32; ++kk)
            umma_f8_warp(tO + j * NP, da + kk * (4096 / 16), dPb + kk * 2, idO, (!first || kk > 0) ? 1u : 0u);
          if (j % BP == BP - 1) umma_commit_warp(&sm->empty[(nbox + j) / BP % NB]);
        }
      };
      if constexpr (C::kPipe) {
        const bool sums = warp != 1;
        if (!sums && a.test_stall && g == 0 && hg == 0) ok = wait(&sm->never, 0);
        for (int si = seg_lo; si < seg_hi && ok; ++si) {
          const int4 sg = a.seg_info[si];
          if (seg_heads(a, sg.x, hg, heads_valid) == 0) continue;
          if (!sums) ok = wait(&sm->q_full, nseg & 1);
          for (int t = sg.y; t < sg.z && ok; ++t, ++ntile, nbox += kNB8) {
            const uint32_t par = (ntile >> 1) & 1;
            if (!sums) {
              // the softmax has read the scores of two tiles ago from this buffer
              if (ntile >= 2) {
                ok = wait(&sm->p_full[ntile & 1], par ^ 1);
                tc_fence_after();
              }
              if (ok) scores(0);
              if (!ok) break;
              if (t + 1 == sg.z) umma_commit_warp(&sm->q_empty);
              umma_commit_warp(&sm->s_full[ntile & 1]);
            } else {
              ok = wait(&sm->p_full[ntile & 1], par);
              const bool first = t == sg.y;
              if (ok && first && nseg > 0) ok = wait(&sm->o_free, (nseg - 1) & 1);
              if (!ok) break;
              weighted_sum(first);
              umma_commit_warp(&sm->pv_done[ntile & 1]);
            }
          }
          if (!ok) break;
          if (sums) umma_commit_warp(&sm->o_done);
          ++nseg;
        }
      } else {
        int early = 0;
        if (a.test_stall && g == 0 && hg == 0) ok = wait(&sm->never, 0);
        for (int si = seg_lo; si < seg_hi && ok; ++si) {
          const int4 sg = a.seg_info[si];
          if (seg_heads(a, sg.x, hg, heads_valid) == 0) continue;
          ok = wait(&sm->q_full, nseg & 1);
          for (int t = sg.y; t < sg.z && ok; ++t) {
            scores(early);
            if (!ok) break;
            if (t + 1 == sg.z) umma_commit_warp(&sm->q_empty);
            umma_commit_warp(&sm->s_full[0]);
            // the next tile's boxes that have landed (a non-blocking probe)
            early = 0;
            if (t + 1 < sg.z) {
              for (int j = 0; j < kNB8; ++j) {
                const uint32_t c = nbox + kNB8 + j;
                if (!__all_sync(0xffffffffu, mbar_test(&sm->full[c % NR], (c / NR) & 1))) break;
                s_box(c % NR, j, tmem + ((ntile + 1) & 1) * N2);
                ++early;
              }
            }
            ok = wait(&sm->p_full[0], ntile & 1);
            const bool first = (t == sg.y);
            if (ok && first && nseg > 0) ok = wait(&sm->o_free, (nseg - 1) & 1);
            if (!ok) break;
            weighted_sum(first);
            nbox += kNB8;
            ++ntile;
          }
          if (!ok) break;
          umma_commit_warp(&sm->o_done);
          ++nseg;
        }
      }
    } else if (lane == 0) {
      constexpr uint32_t idS = idesc_e4m3_f32(128, N2, false, false);
      constexpr uint32_t idO = idesc_e4m3_f32(128, NP, true, false);
      const uint32_t ring_a = smem_u32(ring), q_a = smem_u32(qs), p_a = smem_u32(pbuf);
      const uint64_t dRing = sdesc_sw128(ring_a, 16, 1024), dQ = sdesc_sw128(q_a, 16, 1024);
      const uint64_t dRingMN = sdesc_sw128(ring_a, kBox8, 1024);   // a box read as [tokens (K) x 128 latent dims (M)]
      const uint64_t dP = sdesc_sw128(p_a, 16, 1024);
      auto s_box = [&](uint32_t c, int j, uint32_t tSb) {   // S^T += box j of the tile x its Q box
        const uint64_t da = dRing + (c % NR) * (kBox8 / 16);
        const uint64_t db = dQ + j * (N2 * 128 / 16);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) umma_f8(tSb, da + kk * 2, db + kk * 2, idS, (j | kk) != 0);
      };
      uint32_t nbox = 0, ntile = 0, nseg = 0;
      int early = 0;
      bool ok = true;
      if (a.test_stall && g == 0 && hg == 0) ok = mbar_wait(&sm->never, 0, abort_flag, a.status);
      for (int si = seg_lo; si < seg_hi && ok; ++si) {
        const int4 sg = a.seg_info[si];
        if (seg_heads(a, sg.x, hg, heads_valid) == 0) continue;
        if (!mbar_wait(&sm->q_full, nseg & 1, abort_flag, a.status)) { ok = false; break; }
        for (int t = sg.y; t < sg.z; ++t, ++ntile) {
          const uint32_t tSb = tmem + (ntile & 1) * N2;
          for (int j = early; j < kNB8; ++j) {
            const uint32_t c = nbox + j;
            if (!mbar_wait(&sm->full[c % NR], (c / NR) & 1, abort_flag, a.status)) { ok = false; break; }
            s_box(c, j, tSb);
          }
          if (!ok) break;
          if (t + 1 == sg.z) umma_commit(&sm->q_empty);
          umma_commit(&sm->s_full[0]);
          // the next tile's boxes that have landed (a non-blocking probe)
          early = 0;
          if (t + 1 < sg.z) {
            const uint32_t tSn = tmem + ((ntile + 1) & 1) * N2;
            for (int j = 0; j < kNB8; ++j) {
              const uint32_t c = nbox + kNB8 + j;
              if (!mbar_test(&sm->full[c % NR], (c / NR) & 1)) break;
              s_box(c, j, tSn);
              ++early;
            }
          }
          if (!mbar_wait(&sm->p_full[0], ntile & 1, abort_flag, a.status)) { ok = false; break; }
          const bool first = (t == sg.y);
          if (first && nseg > 0 && !mbar_wait(&sm->o_free, (nseg - 1) & 1, abort_flag, a.status)) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int j = 0; j < kNB8; ++j) {
            const uint32_t slot = (nbox + j) % NR;
            const uint64_t da = dRingMN + slot * (kBox8 / 16);
#pragma unroll
            for (int kk = 0; kk < kTok / 32; ++kk)
              umma_f8(tO + j * NP, da + kk * (4096 / 16), dP + kk * 2, idO, (!first || kk > 0) ? 1u : 0u);
            umma_commit(&sm->empty[slot]);
          }
          nbox += kNB8;
        }
        if (!ok) break;
        umma_commit(&sm->o_done);
        ++nseg;
      }
    }
  } else {
    // ------------------------------ softmax warps ------------------------------
    constexpr int SG = C::kSG, HT = HG / SG;
    const int q4 = warp & 3;
    const int h0 = SG == 1 ? 0 : ((warp - 2) >> 2) * HT;
    const int row = q4 * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(q4 * 32) << 16;
    const int ltid = threadIdx.x - 64;
    const float NEG_INF = -__int_as_float(0x7f800000);
    constexpr float kRaise = BLK ? kRaise8B : kRaise8;
    const float o_mul = BLK ? 1.f / kPScaleB : a.cache_scale / kPScale;
    uint32_t nbox = 0, ntile = 0, nseg = 0;
    bool ok = true;
    for (int si = seg_lo; si < seg_hi; ++si) {
      const int4 sg = a.seg_info[si];
      const int b = sg.x;
      const int L = sg.w;
      const int S0 = a.seq_starts ? a.seq_starts[b] : 0;
      const int hv = seg_heads(a, b, hg, heads_valid);
      if (hv == 0) continue;
      float mul[HT], m[HT], lsum[HT];
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        const int slot = hg * HG + h0 + h;
        mul[h] = (h0 + h < hv && slot < a.H) ? a.qmul[static_cast<int64_t>(b) * a.H + slot] : 0.f;
        m[h] = NEG_INF;
        lsum[h] = 0.f;
      }
      // block scales: this thread's row of a tile has scale sc; the next tile's scale and
      // the page of the tile after it are fetched while a tile is worked on
      float sc = 1.f, sc_next = 1.f;
      int page_next = 0;
      auto scale_page = [&](int t) {   // page of this thread's row in tile t (0 where there is none)
        const int pos = t * kTok + row;
        if (!a.cache.paged || t >= sg.z || pos >= L || pos < S0) return 0;
        return a.cache.block_table[static_cast<int64_t>(b) * a.cache.max_pages_per_seq + pos / a.cache.page_size];
      };
      auto scale_of = [&](int t, int page) {
        const int pos = t * kTok + row;
        if (t >= sg.z || pos >= L || pos < S0) return 1.f;
        int64_t i;
        if (a.cache.paged) {
          if (page < 0 || page >= a.cache.num_pages) {
            report_status(a.status, kStatusRange);
            return 1.f;
          }
          i = (static_cast<int64_t>(page) * a.cache.page_size + pos % a.cache.page_size) >> a.scale_shift;
        } else {
          const int per = (a.cache.capacity + (1 << a.scale_shift) - 1) >> a.scale_shift;
          i = static_cast<int64_t>(b) * per + (pos >> a.scale_shift);
        }
        return a.scales[i];
      };
      if (BLK) {
        sc_next = scale_of(sg.y, scale_page(sg.y));
        page_next = scale_page(sg.y + 1);
      }
      for (int t = sg.y; t < sg.z; ++t, ++ntile) {
        const bool first = (t == sg.y);
        float lg = 0.f, isc = 1.f, offset = 0.f;
        if (BLK) {
          offset = term_offset(t * kTok + row);
          sc = sc_next;
          sc_next = scale_of(t + 1, page_next);
          page_next = scale_page(t + 2);
          if (!(sc >= kScaleMin && sc <= kScaleMax)) {
            report_status(a.status, kStatusRange);
            sc = 1.f;
          }
          lg = __log2f(sc);
          isc = 1.f / sc;
        }
        ok = ok && wait8<BLK>(&sm->s_full[C::kPipe ? ntile & 1 : 0], (C::kPipe ? ntile >> 1 : ntile) & 1, abort_flag, a.status);
        tc_fence_after();
        const uint32_t tS = tmem + (ntile & 1) * N2 + lane_off + h0;
        const int valid = min(kTok, L - t * kTok);
        const bool rv = row < valid && t * kTok + row >= S0;
        auto load16 = [&](int c, float (&x)[16]) {   // score = (hi + lo) * sigma * cache_scale
          uint32_t vh[16], vl[16];
          tmem_ld16(tS + c, vh);
          tmem_ld16(tS + HG + c, vl);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j)
            x[j] = !rv ? NEG_INF
                   : BLK ? fmaf((__uint_as_float(vh[j]) + __uint_as_float(vl[j])) * mul[c + j], sc, lg)
                         : (__uint_as_float(vh[j]) + __uint_as_float(vl[j])) * mul[c + j];
        };
        // block scales: 16 heads a thread, whose scores stay in registers
        static_assert(!BLK || HT == 16, "scores in registers");
        float xs[BLK ? 16 : 1];
        if constexpr (BLK) load16(0, xs);
        auto scores16 = [&](int c, float (&x)[16]) {
          if constexpr (BLK) {
#pragma unroll
            for (int j = 0; j < 16; ++j) x[j] = xs[j];
          } else {
            load16(c, x);
          }
        };
        bool need = first;
#pragma unroll
        for (int c = 0; c < HT; c += 16) {
          float x[16];
          scores16(c, x);
#pragma unroll
          for (int j = 0; j < 16; ++j) need |= x[j] > m[c + j] + kRaise;
        }
        const int par = ntile & 1;
        const int vslot = static_cast<int>(ntile % 3u);
        if (__any_sync(0xffffffffu, need) && lane == 0) atomicOr(&sm->vote[vslot], 1);
        asm volatile("bar.sync 1, %0;" ::"n"(128 * SG) : "memory");
        const bool need_all = sm->vote[vslot] != 0;
        if (ltid == 0) sm->vote[(vslot + 2) % 3] = 0;
        if (need_all) {
#pragma unroll
          for (int c = 0; c < HT; c += 16) {
            float x[16];
            scores16(c, x);
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int k = __reduce_max_sync(0xffffffffu, float_to_ordered(x[j]));
              if (lane == 0) sm->red[par][q4][h0 + c + j] = k;
            }
          }
          asm volatile("bar.sync 1, %0;" ::"n"(128 * SG) : "memory");
          if (C::kPipe && !first) {   // the weighted sum before this tile's may still be adding to O
            ok = ok && wait8<BLK>(&sm->pv_done[(ntile - 1) & 1], ((ntile - 1) >> 1) & 1, abort_flag, a.status);
            ok = __all_sync(0xffffffffu, ok);
            tc_fence_after();
          }
#pragma unroll
          for (int c = 0; c < HT; c += 16) {
            float alpha[16];
            bool rescale = false;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const int h = c + j;
              int k = sm->red[par][0][h0 + h];
              k = max(k, sm->red[par][1][h0 + h]);
              k = max(k, sm->red[par][2][h0 + h]);
              k = max(k, sm->red[par][3][h0 + h]);
              const float tmax = ordered_to_float(k);
              const float mn = fmaxf(m[h], tmax);
              alpha[j] = (m[h] == NEG_INF) ? 0.f : ex2_approx(m[h] - mn);
              rescale |= (mn > m[h]) && !first;
              m[h] = mn;
              lsum[h] *= alpha[j];
            }
            if (rescale) {   // the hi and lo columns of O^T of these heads scale by alpha
#pragma unroll 1
              for (int mc = 0; mc < kNB8; ++mc) {
#pragma unroll
                for (int part = 0; part < C::kTerms; ++part) {
                  uint32_t v[16];
                  const uint32_t col = tO + lane_off + mc * NP + part * HG + h0 + c;
                  tmem_ld16(col, v);
                  tmem_ld_wait();
#pragma unroll
                  for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha[j]);
                  tmem_st16(col, v);
                }
              }
              tmem_st_wait();
            }
          }
        }
        // P' = kPScale exp2(s - m) as e4m3 terms, this thread's token column
        // of P [terms x HG heads x 128 tokens] (K-major, 128-byte swizzle)
        uint8_t* pb = pbuf + (C::kPipe ? (ntile & 1) * C::kPBuf : 0);
        if (C::kPipe && ntile >= 2) {   // the weighted sum of two tiles ago has read this buffer
          ok = ok && wait8<BLK>(&sm->pv_done[ntile & 1], ((ntile >> 1) & 1) ^ 1, abort_flag, a.status);
          ok = __all_sync(0xffffffffu, ok);
        }
#pragma unroll
        for (int c = 0; c < HT; c += 16) {
          float x[16];
          scores16(c, x);
          if constexpr (BLK) {
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              const int h = h0 + c + j;
              const float p0 = rv ? ex2_approx(x[j] - m[c + j]) : 0.f;
              const float p1 = rv ? ex2_approx(x[j + 1] - m[c + j + 1]) : 0.f;
              lsum[c + j] = fmaf(p0, isc, lsum[c + j]);
              lsum[c + j + 1] = fmaf(p1, isc, lsum[c + j + 1]);
              uint32_t term[C::kTerms];
              terms_e4m3x2<C::kTerms>(p0 * kPScaleB, p1 * kPScaleB, offset, term);
#pragma unroll
              for (int k = 0; k < C::kTerms; ++k) {
                pb[sw128_byte(k * HG + h, row)] = static_cast<uint8_t>(term[k]);
                pb[sw128_byte(k * HG + h + 1, row)] = static_cast<uint8_t>(term[k] >> 8);
              }
            }
            continue;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const int h = h0 + c + j;
            const float p = rv ? ex2_approx(x[j] - m[c + j]) : 0.f;
            lsum[c + j] += p;
            uint8_t hi, lo;
            split_e4m3(p * kPScale, hi, lo);
            pb[sw128_byte(h, row)] = hi;
            pb[sw128_byte(HG + h, row)] = lo;
          }
        }
        if (!rv) {   // rows outside [start, L) may hold anything (a NaN code): zero them
#pragma unroll 1
          for (int j = h0 / HT; j < kNB8; j += SG) {
            uint8_t* box = ring + ((nbox + j) % NR) * kBox8 + row * 128;
#pragma unroll
            for (int k = 0; k < 8; ++k) reinterpret_cast<uint4*>(box)[k] = make_uint4(0, 0, 0, 0);
          }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(&sm->p_full[C::kPipe ? ntile & 1 : 0]);
        nbox += kNB8;
      }
      // ---- segment end: the partial (O, m, l)
      ok = ok && wait8<BLK>(&sm->o_done, nseg & 1, abort_flag, a.status);
      tc_fence_after();
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        float v = lsum[h];
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) sm->lred[q4][h0 + h] = v;
        if (SG > 1 && lane == 0 && q4 == 0) sm->mfin[h0 + h] = m[h];
      }
      asm volatile("bar.sync 1, %0;" ::"n"(128 * SG) : "memory");
      const int64_t pbase = (static_cast<int64_t>(hg) * a.max_seg + si) * HG;
      if (ok && ltid < hv) {
        float l = 0.f, mh = NEG_INF;
        if (SG == 1) {
#pragma unroll
          for (int h = 0; h < HT; ++h)
            if (h == ltid) mh = m[h];
        } else {
          mh = sm->mfin[ltid];
        }
        for (int w = 0; w < 4; ++w) l += sm->lred[w][ltid];
        a.ml_part[(pbase + ltid) * 2 + 0] = mh;
        a.ml_part[(pbase + ltid) * 2 + 1] = l;
      }
#pragma unroll 1
      for (int mc = 0; mc < kNB8; ++mc) {
#pragma unroll
        for (int c = 0; c < HT; c += 16) {
          uint32_t vh[16], vl[16], vt[16];
          tmem_ld16(tO + lane_off + mc * NP + h0 + c, vh);
          tmem_ld16(tO + lane_off + mc * NP + HG + h0 + c, vl);
          if (BLK) tmem_ld16(tO + lane_off + mc * NP + 2 * HG + h0 + c, vt);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float hi = __uint_as_float(vh[j]), lo = __uint_as_float(vl[j]);
            const float v = BLK ? fmaf(fmaf(__uint_as_float(vt[j]), 1.f / 32.f, lo), 1.f / 32.f, hi) : hi + lo;
            if (ok && h0 + c + j < hv) a.o_part[(pbase + h0 + c + j) * kDc8 + mc * 128 + row] = v * o_mul;
          }
        }
      }
      tc_fence_before();
      asm volatile("bar.sync 1, %0;" ::"n"(128 * SG) : "memory");
      mbar_arrive(&sm->o_free);
      ++nseg;
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // A wait gave up: copies land and products end before their memory goes. Here every role has left its loop and the
  // flag is settled; a role that ran to its end while another gave up has nobody else to wait for what it issued.
  if (*abort_flag) {
    if (warp == 0 && lane == 0) {
      const uint32_t n = (loaded + BP - 1) / BP;
      for (uint32_t c = n > static_cast<uint32_t>(NB) ? n - NB : 0; c < n; ++c)
        mbar_drain(&sm->full[c % NB], (c / NB) & 1);
      if (loaded_q) mbar_drain(&sm->q_full, (loaded_q - 1) & 1);
    }
    if (warp == 1 || (C::kPipe && warp == C::kThreads / 32 - 1)) {
      if (BLK)
        umma_commit_warp(&sm->drain);
      else if (lane == 0)
        umma_commit(&sm->drain);
      mbar_drain(&sm->drain, 0);
    }
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

template <int HG, bool BLK>
static cudaError_t launch_attn_fp8(const DecodeArgs& a, cudaStream_t st) {
  using C = Dec8Cfg<HG, BLK>;
  auto k = decode_attn_fp8_kernel<HG, BLK>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  prof_begin(st, "decode_attn");
  e = launch_pdl(k, dim3(a.G, a.n_hg), dim3(C::kThreads), C::kSmem, st, 1, a, !BLK);
  prof_end(st);
  return e;
}

}  // namespace gmla
