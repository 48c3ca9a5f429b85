// w4_tc.cuh — the product with 4-bit weights on tcgen05 (included by w4.cu).
//
// y^T = W a^T with M = 128 weight rows, N = BN tokens (16 .. 128), K = 128 codes a
// block, for more tokens than the m16n8k16 kernel is good for. The codes are
// expanded inside the kernel: a code v becomes the exact bf16 integer v - 8, so the
// tensor-core sum of one group is sum (code - 8) a with no rounded weight, and the
// group's scale is applied in fp32 when its accumulator leaves tensor memory.
//
// Roles (one CTA per SM, each working through an equal range of 256-k chunks of the
// row x token tiles laid end to end):
//   * a copy warp streams code boxes (128 rows x 128 bytes = 256 k) and activation
//     boxes (BN tokens x 64 k);
//   * eight expanding warps: thread = row, 32 bytes of codes become 32 columns (64 k) of an A
//     block of 128 k in tensor memory. (Through shared memory, which the MMA would read
//     again, the kernel was bound by shared-memory bandwidth: 530 cycles for 64 k.)
//   * one thread issues the MMAs: a group's blocks accumulate into one of two
//     TMEM buffers;
//   * four warps (eight at BN = 128) promote: acc += scale[row] * buffer, thread = row.
// What bounds it: at BN <= 128 an MMA of M = 128, K = 16 costs a fixed 64 cycles, 256
// cycles for 4 KB of codes, which is 0.7 of the HBM rate at few tokens and the full
// bf16 rate at 128; the expansion (11 instructions and a 16-byte store for 8 codes) and
// the promotion (a load and a fused multiply-add per accumulator and group) run beside it.
// A range that ends inside a tile leaves a partial fp32 tile in the workspace;
// w4_reduce adds those of each split tile in the order of k.
#pragma once

namespace gmla {

namespace {

struct W4TcSmem {
  uint64_t code_full[4], code_empty[4];
  uint64_t full[4], ax_empty[4];   // an A block and its activations: 256 expanding threads and the copy thread arrive
  uint64_t d_full[2], d_free[2];
  uint64_t drain;
  uint32_t tmem;
  int abort;
};

template <int BN>
struct W4TcCfg {
  static constexpr int kEpi = BN == 128 ? 8 : 4;               // promoting warps
  static constexpr int kCols = BN / (kEpi / 4);                // accumulators a thread
  static constexpr int kThreads = 32 * (2 + kEpi + 8);
  static constexpr int kCode = 128 * 128;                      // 256 k
  static constexpr int kX = BN * 256;                          // activations of a block of 128 k: two tiles of 128-byte rows
  static constexpr int kCodeStages = 4, kStages = 3;
  static constexpr int kACols = 64;                            // TMEM columns of an A block (two bf16 each)
  static constexpr int kTmemUsed = 2 * BN + kStages * kACols;
  static constexpr int kTmem = kTmemUsed <= 256 ? 256 : 512;
  static constexpr int kSmem = kCodeStages * kCode + kStages * kX + 1024 + static_cast<int>(sizeof(W4TcSmem));
  static_assert(kTmemUsed <= 512, "tensor memory");
  static_assert(kSmem <= 232448, "shared memory");
};

// First chunk of the range of CTA i, when U chunks are cut into G equal ranges.
__host__ __device__ inline int w4_range(int64_t U, int G, int i) { return static_cast<int>(U * i / G); }

}  // namespace

template <int BN, int MPG>   // MPG: MMAs (16 k) a group: 2, 4 or 8
__global__ void __launch_bounds__(W4TcCfg<BN>::kThreads, 1) w4_tc_kernel(const __grid_constant__ W4TcArgs a) {
  using C = W4TcCfg<BN>;
  constexpr int NC = C::kCodeStages, NS = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* codes = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sx = codes + NC * C::kCode;
  W4TcSmem* sm = reinterpret_cast<W4TcSmem*>(sx + NS * C::kX);
  volatile int* abort_flag = &sm->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NC; ++i) {
      mbar_init(&sm->code_full[i], 1);
      mbar_init(&sm->code_empty[i], 8);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sm->full[i], 257);
      mbar_init(&sm->ax_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm->d_full[i], 1);
      mbar_init(&sm->d_free[i], 32 * C::kEpi);
    }
    mbar_init(&sm->drain, 1);
    sm->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sm->tmem, C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0) griddep_launch_dependents();
  const uint32_t tmem = sm->tmem;          // two accumulators of BN columns, then the A blocks
  const uint32_t tA = tmem + 2 * BN;
  const int n_chunk = a.n_chunk;
  const int64_t U = static_cast<int64_t>(a.row_tiles) * a.tok_tiles * n_chunk;
  const int u_lo = w4_range(U, gridDim.x, blockIdx.x), u_hi = w4_range(U, gridDim.x, blockIdx.x + 1);
  const int n_u = u_hi - u_lo;

  if (warp == 0) {
    // ------------------------------ copies ------------------------------
    if (lane == 0) {
      tma_prefetch_desc(&a.wmap);
      tma_prefetch_desc(&a.xmap);
      const uint64_t pol_w = a.tok_tiles > 1 ? l2_evict_normal() : l2_evict_first(), pol_x = l2_evict_last();
      auto load_w = [&](int i) {   // chunk i of the range
        const int u = u_lo + i, tile = u / n_chunk;
        mbar_arrive_expect_tx(&sm->code_full[i % NC], C::kCode);
        tma_load_2d(&a.wmap, &sm->code_full[i % NC], codes + (i % NC) * C::kCode, (u % n_chunk) * 128,
                    tile / a.tok_tiles * 128, pol_w);
      };
      // the weights: the kernel before this one (w4_prep) neither writes them nor starts this
      // one before all earlier kernels are done, so they are requested before the wait
      int wi = 0, xi = 0;
      for (; wi < n_u && wi < NC; ++wi) load_w(wi);
      griddep_wait();
      bool ok = true;
      for (int i = 0; i < n_u && ok; ++i) {
        const int u = u_lo + i, tile = u / n_chunk, k0 = (u % n_chunk) * kW4Chunk, t0 = tile % a.tok_tiles * BN;
        for (int j = 0; j < 2; ++j, ++xi) {
          const int s = xi % NS;
          if (xi >= NS && !mbar_poll<20>(&sm->ax_empty[s], ((xi / NS) & 1) ^ 1, abort_flag, a.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&sm->full[s], C::kX);
          for (int h = 0; h < 2; ++h)
            tma_load_2d(&a.xmap, &sm->full[s], sx + s * C::kX + h * (C::kX / 2), k0 + j * 128 + h * 64, t0, pol_x);
        }
        if (!ok) break;
        // the code stage that held chunk wi - NC: freed by the expanding warps, which run ahead of the MMAs
        if (wi < n_u) {
          if (!mbar_poll<20>(&sm->code_empty[wi % NC], ((wi / NC) & 1) ^ 1, abort_flag, a.status)) break;
          load_w(wi++);
        }
      }
      if (*abort_flag) {   // let issued copies land before the block exits
        for (int i = wi > NC ? wi - NC : 0; i < wi; ++i) mbar_drain(&sm->code_full[i % NC], (i / NC) & 1);
        for (int i = xi > NS ? xi - NS : 0; i < xi; ++i) mbar_drain(&sm->full[i % NS], (i / NS) & 1);
      }
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer (the whole warp, converged) ------------------------------
    constexpr uint32_t id = idesc_bf16_f32(128, BN, false, false);
    const uint64_t dX = sdesc_sw128(smem_u32(sx), 16, 1024);
    bool ok = true;
    uint32_t grp = 0;                            // groups begun so far
    for (int b = 0; b < 2 * n_u; ++b) {
      const int s = b % NS;
      ok = mbar_poll<0>(&sm->full[s], (b / NS) & 1, abort_flag, a.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t ta = tA + s * C::kACols;
      const uint64_t dx = dX + s * (C::kX / 16);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        if (kk % MPG == 0 && grp >= 2) {   // the buffer was read by the promoting warps
          ok = ok && mbar_poll<0>(&sm->d_free[grp & 1], ((grp >> 1) & 1) ^ 1, abort_flag, a.status);
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
        }
        if (ok)
          umma_bf16_ta_warp(tmem + (grp & 1) * BN, ta + kk * 8, dx + (kk >> 2) * (C::kX / 32) + (kk & 3) * 2, id,
                            kk % MPG != 0 ? 1u : 0u);
        if (kk % MPG == MPG - 1) {
          if (ok) umma_commit_warp(&sm->d_full[grp & 1]);
          ++grp;
        }
      }
      if (!ok) break;
      umma_commit_warp(&sm->ax_empty[s]);
    }
    if (!ok) {
      umma_commit_warp(&sm->drain);
      mbar_drain(&sm->drain, 0);
    }
  } else if (warp < 2 + C::kEpi) {
    // ------------------------------ promotion ------------------------------
    const int q4 = warp & 3;
    const int col0 = ((warp - 2) >> 2) * C::kCols;
    const int row = q4 * 32 + lane;
    const uint32_t t_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + col0;
    constexpr int gpc = 16 / MPG;
    const int n_groups = a.K / a.group;
    griddep_wait();   // y and the partial tiles may still be read by an earlier kernel
    float acc[C::kCols];
#pragma unroll
    for (int j = 0; j < C::kCols; ++j) acc[j] = 0.f;
    const __nv_bfloat16* scales = static_cast<const __nv_bfloat16*>(a.scales);
    // the scales of a chunk's groups (up to 8), one chunk ahead of their use
    uint32_t next[4] = {0, 0, 0, 0};
    auto load_scales = [&](int u) {
      const int r = u / n_chunk / a.tok_tiles * 128 + row, first = (u % n_chunk) * gpc;
      const __nv_bfloat16* p = scales + static_cast<int64_t>(r < a.N ? r : 0) * n_groups + first;
      if (a.vec_scales) {
        if (gpc == 8) {
          const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
          next[0] = v.x, next[1] = v.y, next[2] = v.z, next[3] = v.w;
        } else if (gpc == 4) {
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
          next[0] = v.x, next[1] = v.y;
        } else {
          next[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = 2 * j < gpc && first + 2 * j < n_groups ? __bfloat16_as_ushort(p[2 * j]) : 0;
          const uint32_t hi = 2 * j < gpc && first + 2 * j + 1 < n_groups ? __bfloat16_as_ushort(p[2 * j + 1]) : 0;
          next[j] = lo | (hi << 16);
        }
      }
    };
    if (n_u > 0) load_scales(u_lo);
    uint32_t grp = 0;
    bool ok = true;
    int seg_lo = u_lo;   // first chunk of the current segment
    for (int u = u_lo; u < u_hi && ok; ++u) {
      uint32_t cur[4] = {next[0], next[1], next[2], next[3]};
      if (u + 1 < u_hi) load_scales(u + 1);
#pragma unroll 1
      for (int g = 0; g < gpc; ++g, ++grp) {
        const uint32_t w = g < 4 ? (g < 2 ? cur[0] : cur[1]) : (g < 6 ? cur[2] : cur[3]);
        const float s = __uint_as_float((g & 1) ? (w & 0xffff0000u) : (w << 16));
        const uint32_t buf = grp & 1;
        ok = mbar_poll<20>(&sm->d_full[buf], (grp >> 1) & 1, abort_flag, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < C::kCols; c += 16) {
          uint32_t v[16];
          tmem_ld16(t_base + buf * BN + c, v);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[c + j] = fmaf(s, __uint_as_float(v[j]), acc[c + j]);
        }
        tc_fence_before();
        mbar_arrive(&sm->d_free[buf]);
      }
      if (!ok) break;
      const int tile = u / n_chunk;
      if (u + 1 == u_hi || (u + 1) % n_chunk == 0) {   // segment end
        const int r = tile / a.tok_tiles * 128 + row, t0 = tile % a.tok_tiles * BN + col0;
        const bool whole = seg_lo == tile * n_chunk && u + 1 == (tile + 1) * n_chunk;
        if (whole) {
          __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + r;
#pragma unroll
          for (int j = 0; j < C::kCols; ++j)
            if (r < a.N && t0 + j < a.T) y[static_cast<int64_t>(t0 + j) * a.N] = __float2bfloat16_rn(acc[j]);
        } else {       // the CTA's first segment in slot 0, its last in slot 1
          float* p = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + (seg_lo == u_lo ? 0 : 1)) * BN * 128 + row;
#pragma unroll
          for (int j = 0; j < C::kCols; ++j) p[(col0 + j) * 128] = acc[j];
        }
#pragma unroll
        for (int j = 0; j < C::kCols; ++j) acc[j] = 0.f;
        seg_lo = u + 1;
      }
    }
  } else {
    // ------------------------------ expansion ------------------------------
    const int wg = (warp - 2 - C::kEpi) >> 2;                    // half of a block
    const int row = (warp & 3) * 32 + lane;                      // a warp reaches the TMEM lanes of its quarter
    const uint32_t t_dst = tA + (static_cast<uint32_t>((warp & 3) * 32) << 16) + wg * 32;
    const uint32_t sw = row & 7;
    const uint32_t eight = 0x43084308u;                          // (136, 136)
    bool ok = true;
    for (int i = 0; i < n_u && ok; ++i) {
      ok = mbar_poll<20>(&sm->code_full[i % NC], (i / NC) & 1, abort_flag, a.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint8_t* src = codes + (i % NC) * C::kCode + row * 128;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int j = 2 * h + wg, b = 2 * i + h, s = b % NS;     // 64 k number j of the chunk, half wg of block b
        uint4 w[2];
        w[0] = *reinterpret_cast<const uint4*>(src + (((2 * j) ^ sw) << 4));
        w[1] = *reinterpret_cast<const uint4*>(src + (((2 * j + 1) ^ sw) << 4));
        if (h == 1) {   // this warp's codes of the chunk are in registers
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->code_empty[i % NC]);
        }
        if (b >= NS) {
          ok = mbar_poll<20>(&sm->ax_empty[s], ((b / NS) & 1) ^ 1, abort_flag, a.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        tc_fence_after();
        const uint32_t word[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
        for (int k = 0; k < 8; k += 4) {
          uint32_t p[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            p[q] = w4_pair(word[k + (q >> 2)], q & 3);
            asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(p[q]) : "r"(eight));
          }
          tmem_st16(t_dst + s * C::kACols + k * 4, p);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sm->full[s]);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
  }
}

// ---------------------------------------------------------------------------
// y of the tiles whose chunks lie in more than one CTA's range: the partial tiles in
// the order of k. Grid (row x token tiles, BN / 8 token octets); thread = row.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(128) w4_reduce_kernel(W4ReduceArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t U = static_cast<int64_t>(a.tiles) * a.n_chunk;
  const int tile = blockIdx.x;
  const int64_t u0 = static_cast<int64_t>(tile) * a.n_chunk, u1 = u0 + a.n_chunk;
  // CTA of chunk u: the largest i with U i / G <= u
  const int i0 = static_cast<int>(((u0 + 1) * a.G - 1) / U), i1 = static_cast<int>((u1 * a.G - 1) / U);
  if (i0 == i1) return;   // one CTA had the whole tile and wrote y
  const int r = threadIdx.x, row = tile / a.tok_tiles * 128 + r;
  const int c0 = blockIdx.y * 8, t0 = tile % a.tok_tiles * a.BN + c0;
  float acc[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) acc[j] = 0.f;
  for (int i = i0; i <= i1; ++i) {
    const int slot = w4_range(U, a.G, i) >= u0 ? 0 : 1;
    const float* p = a.part + ((static_cast<int64_t>(i) * 2 + slot) * a.BN + c0) * 128 + r;
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] += __ldcg(p + j * 128);
  }
  if (row < a.N) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (t0 + j < a.T)
        static_cast<__nv_bfloat16*>(a.y)[static_cast<int64_t>(t0 + j) * a.N + row] = __float2bfloat16_rn(acc[j]);
  }
}

}  // namespace gmla
