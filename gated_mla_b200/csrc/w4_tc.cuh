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
//   * one warp streams code boxes (128 rows x 128 bytes = 256 k), another the activations
//     (BN tokens x 128 k, stored by w4_prep as the image of the swizzled shared-memory
//     tiles: one bulk copy). Together in one thread, with its waits, they took 950 cycles a block;
//   * eight expanding warps: thread = row, 32 bytes of codes become 32 columns (64 k) of an A
//     block of 128 k in tensor memory. (Through shared memory, which the MMA would read
//     again, the kernel was bound by shared-memory bandwidth: 530 cycles for 64 k.)
//   * two warps issue the MMAs, of alternate blocks, into accumulators of their own: a wait on
//     a barrier costs about 250 cycles even when it is complete, an MMA of this size 45
//     (one issuing warp: 1040 cycles a block of 128 k);
//   * four warps (eight from BN = 64 on) promote: acc += scale[row] * buffer, thread = row.
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
  uint64_t full[4], ax_empty[4];   // an A block and its activations: the expanding threads and a copy thread arrive
  uint64_t d_full[4], d_free[4];
  uint64_t drain[2];
  uint32_t tmem;
  int abort;
};

template <int BN>
struct W4TcCfg {
  static constexpr int kEpi = BN >= 64 ? 8 : 4;                // promoting warps
  static constexpr int kCols = BN / (kEpi / 4);                // accumulators a thread
  static constexpr int kExp = BN == 128 ? 4 : 8;               // expanding warps (with 8 at BN = 128 the sums would spill)
  static constexpr int kThreads = 32 * (4 + kEpi + kExp);
  static constexpr int kCode = 128 * 128;                      // 256 k
  static constexpr int kX = BN * 256;                          // activations of a block of 128 k: two tiles of 128-byte rows
  static constexpr int kCodeStages = 4, kStages = 3;
  static constexpr int kACols = 64;                            // TMEM columns of an A block (two bf16 each)
  static constexpr int kBufs = BN == 128 ? 1 : 2;              // accumulators of an issuing warp
  static constexpr int kTmemUsed = 2 * kBufs * BN + kStages * kACols;
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
      mbar_init(&sm->code_empty[i], C::kExp);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&sm->full[i], 32 * C::kExp + 1);
      mbar_init(&sm->ax_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm->d_full[i], 1);
      mbar_init(&sm->d_free[i], 32 * C::kEpi);
    }
    mbar_init(&sm->drain[0], 1);
    mbar_init(&sm->drain[1], 1);
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
  const uint32_t tmem = sm->tmem;          // the accumulators of BN columns, then the A blocks
  const uint32_t tA = tmem + 2 * C::kBufs * BN;
  constexpr int GPB = 8 / MPG;             // groups a block: group g of block b is number (b >> 1) * GPB + g of its warp
  const int n_chunk = a.n_chunk;
  const int64_t U = static_cast<int64_t>(a.row_tiles) * a.tok_tiles * n_chunk;
  const int u_lo = w4_range(U, gridDim.x, blockIdx.x), u_hi = w4_range(U, gridDim.x, blockIdx.x + 1);
  const int n_u = u_hi - u_lo;
  // the range's first tile and its first chunk there (counted up from here: a division
  // in a thread that issues alone costs as much as a copy)
  const int tile0 = u_lo / n_chunk, ch0 = u_lo - tile0 * n_chunk;
  const int rt0 = tile0 / a.tok_tiles, tt0 = tile0 - rt0 * a.tok_tiles;

  if (warp == 0) {
    // ------------------------------ codes ------------------------------
    if (lane == 0) {
      tma_prefetch_desc(&a.wmap);
      const uint64_t pol_w = a.tok_tiles > 1 ? l2_evict_normal() : l2_evict_first();
      // the weights: the kernel before this one (w4_prep) neither writes them nor starts this
      // one before all earlier kernels are done, so they are requested without a wait
      int i = 0, ch = ch0, tt = tt0, row = rt0 * 128;
      for (; i < n_u; ++i) {
        const int s = i % NC;
        if (i >= NC && !mbar_poll<20>(&sm->code_empty[s], ((i / NC) & 1) ^ 1, abort_flag, a.status)) break;
        mbar_arrive_expect_tx(&sm->code_full[s], C::kCode);
        tma_load_2d(&a.wmap, &sm->code_full[s], codes + s * C::kCode, ch * 128, row, pol_w);
        if (++ch == n_chunk) {
          ch = 0;
          if (++tt == a.tok_tiles) tt = 0, row += 128;
        }
      }
      if (*abort_flag)   // let issued copies land before the block exits
        for (int c = i > NC ? i - NC : 0; c < i; ++c) mbar_drain(&sm->code_full[c % NC], (c / NC) & 1);
    }
  } else if (warp == 3) {
    // ------------------------------ activations ------------------------------
    if (lane == 0) {
      const uint64_t pol_x = l2_evict_last();
      griddep_wait();
      int b = 0, s = 0, tt = tt0, left = 2 * (n_chunk - ch0);   // blocks left in the tile
      const uint8_t* x = static_cast<const uint8_t*>(a.x);
      const uint8_t* src = x + (static_cast<int64_t>(tt0) * n_chunk + ch0) * 2 * C::kX;
      for (; b < 2 * n_u; ++b) {
        if (b >= NS && !mbar_poll<0>(&sm->ax_empty[s], ((b / NS) & 1) ^ 1, abort_flag, a.status)) break;
        mbar_arrive_expect_tx(&sm->full[s], C::kX);
        bulk_load(sx + s * C::kX, src, C::kX, &sm->full[s], pol_x);
        src += C::kX;
        if (--left == 0) {   // the next tile: its tokens follow, or the first ones again
          left = 2 * n_chunk;
          if (++tt == a.tok_tiles) tt = 0, src = x;
        }
        if (++s == NS) s = 0;
      }
      if (*abort_flag)
        for (int c = b > NS ? b - NS : 0; c < b; ++c) mbar_drain(&sm->full[c % NS], (c / NS) & 1);
    }
  } else if (warp <= 2) {
    // ------------------------------ MMA issuers (whole warps, converged) ------------------------------
    constexpr uint32_t id = idesc_bf16_f32(128, BN, false, false);
    const uint64_t dX = sdesc_sw128(smem_u32(sx), 16, 1024);
    const int me = warp - 1;
    bool ok = true;
    uint32_t n = 0;                              // groups begun by this warp
    for (int b = me; b < 2 * n_u && ok; b += 2) {
      const int s = b % NS;
      ok = mbar_poll<0>(&sm->full[s], (b / NS) & 1, abort_flag, a.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc_fence_after();
      const uint32_t ta = tA + s * C::kACols;
      const uint64_t dx = dX + s * (C::kX / 16);
#pragma unroll
      for (int g = 0; g < GPB; ++g, ++n) {
        const int buf = me * C::kBufs + n % C::kBufs;
        if (n >= C::kBufs) {   // the accumulator was read by the promoting warps
          ok = mbar_poll<0>(&sm->d_free[buf], (n / C::kBufs & 1) ^ 1, abort_flag, a.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
        }
#pragma unroll
        for (int k = 0; k < MPG; ++k) {
          const int q = g * MPG + k;             // 16-k step of the block
          umma_bf16_ta_warp(tmem + buf * BN, ta + q * 8, dx + (q >> 2) * (C::kX / 32) + (q & 3) * 2, id, k != 0 ? 1u : 0u);
        }
        umma_commit_warp(&sm->d_full[buf]);
      }
      if (ok) umma_commit_warp(&sm->ax_empty[s]);
    }
    if (!ok) {
      umma_commit_warp(&sm->drain[me]);
      mbar_drain(&sm->drain[me], 0);
    }
  } else if (warp < 4 + C::kEpi) {
    // ------------------------------ promotion ------------------------------
    const int q4 = warp & 3;
    const int col0 = ((warp - 4) >> 2) * C::kCols;
    const int row = q4 * 32 + lane;
    const uint32_t t_base = tmem + (static_cast<uint32_t>(q4 * 32) << 16) + col0;
    constexpr int gpc = 16 / MPG;
    const int n_groups = a.K / a.group;
    griddep_wait();   // y and the partial tiles may still be read by an earlier kernel
    float acc[C::kCols];
#pragma unroll
    for (int j = 0; j < C::kCols; ++j) acc[j] = 0.f;
    const __nv_bfloat16* scales = static_cast<const __nv_bfloat16*>(a.scales);
    // the scales of a chunk's groups (up to 8), one chunk ahead of their use; at 64 columns a
    // thread, where registers are short and groups slow, each one a group ahead
    constexpr bool kOneScale = C::kCols == 64;
    uint32_t next[kOneScale ? 1 : 4];
    auto load_scales = [&](int rt, int ch) {
      const int r = rt * 128 + row, first = ch * gpc;
      const __nv_bfloat16* p = scales + static_cast<int64_t>(r < a.N ? r : 0) * n_groups + first;
      if constexpr (!kOneScale) {
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
          return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t lo = 2 * j < gpc && first + 2 * j < n_groups ? __bfloat16_as_ushort(p[2 * j]) : 0;
          const uint32_t hi = 2 * j < gpc && first + 2 * j + 1 < n_groups ? __bfloat16_as_ushort(p[2 * j + 1]) : 0;
          next[j] = lo | (hi << 16);
        }
      }
    };
    auto load_one = [&](int rt, int grp) {       // groups behind K scale nothing
      const int r = rt * 128 + row;
      next[0] = grp < n_groups
                    ? __bfloat16_as_ushort(__ldg(scales + static_cast<int64_t>(r < a.N ? r : 0) * n_groups + grp))
                    : 0;
    };
    int rt = rt0, tt = tt0, ch = ch0;      // of the current chunk
    if (n_u > 0) {
      load_scales(rt, ch);
      if (kOneScale) load_one(rt, ch * gpc);
    }
    uint32_t grp = 0;
    bool ok = true;
    int seg_lo = u_lo;   // first chunk of the current segment
    for (int u = u_lo; u < u_hi && ok; ++u) {
      uint32_t cur[kOneScale ? 1 : 4];
      if constexpr (!kOneScale) cur[0] = next[0], cur[1] = next[1], cur[2] = next[2], cur[3] = next[3];
      const bool tile_end = ch + 1 == n_chunk;
      const int rt_next = tile_end && tt + 1 == a.tok_tiles ? rt + 1 : rt;
      if (u + 1 < u_hi) load_scales(rt_next, tile_end ? 0 : ch + 1);
#pragma unroll 1
      for (int g = 0; g < gpc; ++g, ++grp) {
        float s;
        if constexpr (kOneScale) {
          s = __uint_as_float(next[0] << 16);
          if (g + 1 < gpc)
            load_one(rt, ch * gpc + g + 1);
          else if (u + 1 < u_hi)
            load_one(rt_next, tile_end ? 0 : (ch + 1) * gpc);
        } else {
          const uint32_t w = g < 4 ? (g < 2 ? cur[0] : cur[1]) : (g < 6 ? cur[2] : cur[3]);
          s = __uint_as_float((g & 1) ? (w & 0xffff0000u) : (w << 16));
        }
        const uint32_t blk = grp / GPB, n = (blk >> 1) * GPB + grp % GPB;
        const uint32_t buf = (blk & 1) * C::kBufs + n % C::kBufs;
        ok = mbar_poll<20>(&sm->d_full[buf], n / C::kBufs & 1, abort_flag, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        constexpr int W = C::kCols == 32 ? 32 : 16;          // columns a wait (96 registers a thread at 64 columns)
#pragma unroll
        for (int c = 0; c < C::kCols; c += W) {
          uint32_t v[W / 16][16];
#pragma unroll
          for (int i = 0; i < W / 16; ++i) tmem_ld16(t_base + buf * BN + c + 16 * i, v[i]);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < W; ++j) acc[c + j] = fmaf(s, __uint_as_float(v[j / 16][j % 16]), acc[c + j]);
        }
        tc_fence_before();
        mbar_arrive(&sm->d_free[buf]);
      }
      if (!ok) break;
      if (u + 1 == u_hi || tile_end) {   // segment end
        const int r = rt * 128 + row, t0 = tt * BN + col0;
        const bool whole = tile_end && u - seg_lo == ch;
        if (whole) {
          __nv_bfloat16* y = static_cast<__nv_bfloat16*>(a.y) + static_cast<int64_t>(t0) * a.N + r;
          const int left = r < a.N ? a.T - t0 : 0;
#pragma unroll
          for (int j = 0; j < C::kCols; ++j) {
            if (j < left) *y = __float2bfloat16_rn(acc[j]);
            y += a.N;
          }
        } else {       // the CTA's first segment in slot 0, its last in slot 1
          float* p = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + (seg_lo == u_lo ? 0 : 1)) * BN * 128 + row;
#pragma unroll
          for (int j = 0; j < C::kCols; ++j) p[(col0 + j) * 128] = acc[j];
        }
#pragma unroll
        for (int j = 0; j < C::kCols; ++j) acc[j] = 0.f;
        seg_lo = u + 1;
      }
      if (tile_end) {
        ch = 0;
        if (++tt == a.tok_tiles) tt = 0, ++rt;
      } else {
        ++ch;
      }
    }
  } else {
    // ------------------------------ expansion ------------------------------
    constexpr int kHalves = 8 / C::kExp;                         // 64-k halves of a block a thread expands
    const int h0 = C::kExp == 8 ? (warp - 4 - C::kEpi) >> 2 : 0;
    const int row = (warp & 3) * 32 + lane;                      // a warp reaches the TMEM lanes of its quarter
    const uint32_t t_dst = tA + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t sw = row & 7;
    const uint32_t eight = 0x43084308u;                          // (136, 136)
    bool ok = true;
    for (int i = 0; i < n_u && ok; ++i) {
      ok = mbar_poll<20>(&sm->code_full[i % NC], (i / NC) & 1, abort_flag, a.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint8_t* src = codes + (i % NC) * C::kCode + row * 128;
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const int b = 2 * i + blk, s = b % NS;
        uint4 w[kHalves][2];
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            w[h][j] = *reinterpret_cast<const uint4*>(src + (((4 * blk + 2 * (h0 + h) + j) ^ sw) << 4));
        if (blk == 1) {   // this warp's codes of the chunk are in registers
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm->code_empty[i % NC]);
        }
        if (b >= NS) {
          ok = mbar_poll<20>(&sm->ax_empty[s], ((b / NS) & 1) ^ 1, abort_flag, a.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t word[4] = {w[h][j].x, w[h][j].y, w[h][j].z, w[h][j].w};
            uint32_t p[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              p[q] = w4_pair(word[q >> 2], q & 3);
              asm("sub.rn.bf16x2 %0, %0, %1;" : "+r"(p[q]) : "r"(eight));
            }
            tmem_st16(t_dst + s * C::kACols + (h0 + h) * 32 + j * 16, p);
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
