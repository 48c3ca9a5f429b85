// append.cu — new latent rows into an E4M3 cache that holds one scale for every
// block of 2^k token rows (k <= 7, within a page).
//
//   scale = 2^E, E the smallest integer with max |c| over the block <= 448 * 2^E,
//           kept within [-32, 32] (the range gmla_decode covers)
//   code  = E4M3(c / scale), round to nearest even, saturating at +-448
//
// A power of two costs an E4M3 code nothing (the format keeps its relative
// precision over its whole normal range) and makes a later change of scale exact:
// when rows are appended to a block that already holds some and the scale has to
// grow, the held codes are multiplied by old / new scale and rounded again, which
// only changes those that fall below E4M3's normal range.
//
// Bound by HBM for prompts (1024 B read and 512 B written a row), by latency for
// decode steps (64 single rows 6.4 us, 7 prompts of 19600 rows in all 14.4 us, 0.32 of the HBM rate). The
// new rows of a sequence are consecutive, so a block's new rows
// are one run of `latents` rows. The first of them ("leader") stands for the block:
// a unit (one warp for blocks of up to 8 rows, else a CTA of 8 warps) looks through
// a window of token rows for leaders and handles each leader's block alone, its rows
// held in registers between the maximum and the rounding. No two units touch one
// block, so there is nothing to order between them.
#include "common.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace gmla {

namespace {

constexpr int kAppendDc = 512;   // latent width: 16 elements a lane

// Smallest E with top <= 448 * 2^E, within [-32, 32] (448 = 0.875 * 2^9).
__device__ __forceinline__ int block_exponent(float top) {
  if (!(top > 0.f)) return -32;
  if (top > 3.0e38f) return 32;
  const uint32_t u = __float_as_uint(top);
  const int be = static_cast<int>(u >> 23);                       // top = 1.f * 2^(be - 127), subnormals far below -32
  const int e = be - 126 - 9 + ((u & 0x7fffffu) > 0x600000u);     // fraction above 1.75 = 2 * 0.875: one more
  return max(-32, min(32, e));
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
         (static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3)) << 16);
}

// Last sequence whose offset cu[b] is not above t, given cu[0] <= t < cu[B]:
// a 32-way search by one warp (two or three rounds of loads).
__device__ __forceinline__ int find_seq(const int32_t* cu, int B, int t, int lane) {
  int lo = 0, hi = B;   // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step;
    const unsigned above = __ballot_sync(0xffffffffu, i >= hi || cu[i] > t);
    const int k = __ffs(above) - 1;   // the last lane's i is >= hi, so there is one
    const int nlo = lo + k * step;
    hi = min(hi, nlo + step);
    lo = nlo;
  }
  return lo;
}

}  // namespace

// WPL warps a unit, RPW rows a warp (the block has up to WPL * RPW rows). Where few rows are held, four CTAs
// share an SM (7 prompts, blocks of 16: 14.4 us, with 74 registers and three CTAs 17).
template <int WPL, int RPW>
__global__ void __launch_bounds__(256, RPW <= 2 ? 4 : (RPW <= 4 ? 2 : 1)) cache_append_kernel(AppendArgs a) {
  __shared__ float s_top[8];
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int unit = WPL == 1 ? blockIdx.x * 8 + warp : blockIdx.x;
  const int w = WPL == 1 ? 0 : warp;
  const int blk = a.scale_block;
  int t = unit * a.window;
  // one token a sequence, as in a decode step: row t is sequence t's. The offsets that say
  // so are fetched together, and the row meanwhile
  const int guess = min(t, a.B - 1);
  const int cu_end = a.cu[a.B], cu_0 = a.cu[0], cu_g = a.cu[guess], cu_g1 = a.cu[guess + 1];
  if (w == 0 && t < a.T)
    prefetch_l2(static_cast<const __nv_bfloat16*>(a.latents) + static_cast<int64_t>(t) * a.stride + lane * 16);
  if (unit == 0 && w == 0 && lane == 0 && cu_end > a.T) report_status(a.status, kStatusRange);
  const int total = min(cu_end, a.T);
  const int t_end = min(t + a.window, total);
  if (t >= t_end || t < cu_0) return;   // uniform over the unit
  int b = t >= cu_g && t < cu_g1 ? guess : find_seq(a.cu, a.B, t, lane);
  const CacheView& cv = a.cache;
  const int limit = cache_limit(cv);
  uint8_t* codes = static_cast<uint8_t*>(cv.data);
  while (t < t_end) {
    const int c0 = a.cu[b], c1 = min(a.cu[b + 1], a.T);
    if (t >= c1) {   // the next sequence that has new rows
      if (++b >= a.B) break;
      continue;
    }
    const int len = a.seq_lens[b];
    const int past = len - (a.cu[b + 1] - c0);      // rows held before this call
    if (t < c0 || past < 0 || len > limit || b >= cv.batch) {
      if (lane == 0 && w == 0) report_status(a.status, kStatusRange);
      t = max(c1, t + 1);
      continue;
    }
    const int pos = past + (t - c0);
    const int off = pos % blk;
    const int run = min(blk - off, c1 - t);          // new rows of this block from t on
    if (t != c0 && off != 0) {                       // not a leader: an earlier unit has this block
      t += run;
      continue;
    }
    // the block's first row and scale
    const int p0 = pos - off;
    int64_t row0 = -1, si = 0;
    if (!cv.paged) {
      row0 = static_cast<int64_t>(b) * cv.capacity + p0;
      si = static_cast<int64_t>(b) * ((cv.capacity + blk - 1) / blk) + p0 / blk;
    } else {
      const int page = cv.block_table[static_cast<int64_t>(b) * cv.max_pages_per_seq + p0 / cv.page_size];
      if (page >= 0 && page < cv.num_pages) {
        row0 = static_cast<int64_t>(page) * cv.page_size + p0 % cv.page_size;
        si = row0 / blk;
      }
    }
    if (row0 < 0) {
      if (lane == 0 && w == 0) report_status(a.status, kStatusRange);
      t += run;
      continue;
    }
    const float was = off > 0 ? a.scales[si] : 0.f;
    if (off > 0 && !(was >= kScaleMin && was <= kScaleMax)) {   // the held codes mean nothing: no scale would mend them
      if (lane == 0 && w == 0) report_status(a.status, kStatusRange);
      t += run;
      continue;
    }
    // rows r = w + WPL * i of the block: new ones off <= r < off + run
    uint4 x[RPW][2];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const int r = w + WPL * i;
      x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
      if (r >= off && r < off + run) {
        const uint4* src = reinterpret_cast<const uint4*>(
            static_cast<const __nv_bfloat16*>(a.latents) + (static_cast<int64_t>(t) + r - off) * a.stride + lane * 16);
        x[i][0] = src[0];
        x[i][1] = src[1];
      }
    }
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t u[4] = {x[i][h].x, x[i][h].y, x[i][h].z, x[i][h].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(u[j] << 16)), fabsf(__uint_as_float(u[j] & 0xffff0000u))));
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (WPL > 1) {
      if (lane == 0) s_top[w] = top;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < WPL; ++i) top = fmaxf(top, s_top[i]);
      __syncthreads();   // every warp has read the held scale and the maxima
    } else {
      __syncwarp();
    }
    float scale = __uint_as_float(static_cast<uint32_t>(block_exponent(top) + 127) << 23);
    const bool grow = off > 0 && scale > was;
    if (off > 0 && was >= scale) scale = was;
    // 1 / scale: exact for the powers of two written here, and a division where a held scale is none
    const bool pow2 = (__float_as_uint(scale) & 0x7fffffu) == 0;
    const float mul = 1.f / scale;
    if (lane == 0 && w == 0 && (off == 0 || scale != was)) a.scales[si] = scale;
    uint8_t* dst = codes + row0 * kAppendDc + lane * 16;
    if (grow) {
      const float ratio = was / scale;
#pragma unroll 4
      for (int r = w; r < off; r += WPL) {
        uint4* p = reinterpret_cast<uint4*>(dst + static_cast<int64_t>(r) * kAppendDc);
        const uint4 old = *p;
        const uint32_t u[4] = {old.x, old.y, old.z, old.w};
        uint32_t n[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float f[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(u[j] >> (8 * k)), __NV_E4M3);
            f[k] = __half2float(__half(h)) * ratio;
          }
          n[j] = e4m3x4(f[0], f[1], f[2], f[3]);
        }
        *p = make_uint4(n[0], n[1], n[2], n[3]);
      }
    }
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
      const int r = w + WPL * i;
      if (r >= off && r < off + run) {
        uint32_t n[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t u[4] = {x[i][h].x, x[i][h].y, x[i][h].z, x[i][h].w};
          float f[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float lo = __uint_as_float(u[j] << 16), hi = __uint_as_float(u[j] & 0xffff0000u);
            f[2 * j] = pow2 ? lo * mul : lo / scale;
            f[2 * j + 1] = pow2 ? hi * mul : hi / scale;
          }
          n[2 * h] = e4m3x4(f[0], f[1], f[2], f[3]);
          n[2 * h + 1] = e4m3x4(f[4], f[5], f[6], f[7]);
        }
        *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(r) * kAppendDc) = make_uint4(n[0], n[1], n[2], n[3]);
      }
    }
    t += run;
  }
}

cudaError_t launch_cache_append(AppendArgs a, int num_sms, cudaStream_t st) {
  // A unit's window: enough units for about four CTAs an SM, and no more rows than
  // keep the leaders of a window few
  const bool warp_unit = a.scale_block <= 8;
  const int units_wanted = num_sms * 4 * (warp_unit ? 8 : 1);
  a.window = (a.T + units_wanted - 1) / units_wanted;
  const int units = (a.T + a.window - 1) / a.window;
  const dim3 grid(warp_unit ? (units + 7) / 8 : units), block(256);
  prof_begin(st, "cache_append");
  cudaError_t e;
  switch (a.scale_block) {
    case 1: e = launch_pdl(cache_append_kernel<1, 1>, grid, block, 0, st, 1, a); break;
    case 2: e = launch_pdl(cache_append_kernel<1, 2>, grid, block, 0, st, 1, a); break;
    case 4: e = launch_pdl(cache_append_kernel<1, 4>, grid, block, 0, st, 1, a); break;
    case 8: e = launch_pdl(cache_append_kernel<1, 8>, grid, block, 0, st, 1, a); break;
    case 16: e = launch_pdl(cache_append_kernel<8, 2>, grid, block, 0, st, 1, a); break;
    case 32: e = launch_pdl(cache_append_kernel<8, 4>, grid, block, 0, st, 1, a); break;
    case 64: e = launch_pdl(cache_append_kernel<8, 8>, grid, block, 0, st, 1, a); break;
    default: e = launch_pdl(cache_append_kernel<8, 16>, grid, block, 0, st, 1, a); break;
  }
  prof_end(st);
  return e;
}

}  // namespace gmla
