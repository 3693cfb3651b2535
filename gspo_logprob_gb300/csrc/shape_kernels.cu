// Logit shaping (penalties, biases, allow masks, temperature) and the selected
// log-prob under the shaped distribution, with its gradient.
//
// For row i with history h (its first prompt_len tokens the prompt, the rest
// the output), c_j the count of j in the output part:
//   z1 = z / theta if z > 0 else z theta      (j anywhere in the history)
//   z2 = z1 - frequency c_j - presence [c_j > 0] + bias_j
//   z'_j = z2 / T, -inf where the row's allow mask has a 0 bit
// and, with p = softmax(z'),
//   logp = z'_y - LSE(z'),  d logp / d z_j = ([j = y] - p_j) d z'_j / d z_j.
//
// One kernel serves the three calls.  A CTA owns a range of columns for a block
// of rows and keeps the counts of its columns in shared memory: one word per
// column (output count, prompt flag, bias entry) and one bit per column that
// says whether the word is in use, so that eight untouched columns cost one
// byte load.  Rows whose history is that of the row before plus some tokens
// (consecutive rows of a training sequence) only add those tokens; other rows
// rebuild the words by a scan of their history.
//
// Columns are cut into segments of 1024, each the work of one warp: 4 chunks of
// 256 columns, lane l holding columns 8l..8l+7 of a chunk.  The log-prob keeps
// one (max, sum) per row and segment, so its bits depend on V alone: not on the
// columns per CTA, the rows per CTA or the other rows of the batch.
#include <cuda_bf16.h>

#include "internal.h"
#include "ptx.cuh"

namespace gh {
namespace {

constexpr int SH_THREADS = 256;
constexpr int SH_WARPS = SH_THREADS / 32;
constexpr int SH_CHUNKS = 4;                     // 16-byte loads a lane has in flight
constexpr int SH_SEG = SH_CHUNKS * 256;          // columns per warp segment
constexpr int SH_MAX_COLS = 16384;               // columns per CTA: 64 KB of words, three CTAs per SM
constexpr int SH_MAX_ROWS = 32;                  // rows per CTA (one lane each in the set-up)
constexpr float SH_LOG2E = 1.4426950408889634f;

// the word of a column: bits 0-19 output count, 20 seen in the prompt, 21-31
// bias entry + 1 of the row's list
constexpr uint32_t SH_COUNT = SHAPE_MAX_HIST;
constexpr uint32_t SH_PROMPT = 1u << 20;
constexpr int SH_BIAS_SHIFT = 21;
static_assert(SH_COUNT + 1 == SH_PROMPT && SHAPE_MAX_BIAS == (1 << (32 - SH_BIAS_SHIFT)) - 1, "word layout");

enum { SHAPE_OUT = 0, SHAPE_LOGP = 1, SHAPE_GRAD = 2 };

// how the words go from the row before to this one
enum { TAB_NONE = 0, TAB_KEEP = 1, TAB_ADD1 = 2, TAB_ADD = 3, TAB_BUILD = 4 };  // NONE: the row uses no words

struct ShRow {
  long long begin;  // first history token
  int len, plen;    // history tokens, of which plen are the prompt's
  int bias_b, bias_e;
  int allow;        // row of allow_bits or -1
  int y;
  int tab;          // TAB_*
  int add_from;     // TAB_ADD: history tokens [add_from, len) are new; TAB_ADD1: the token itself
  float rep, inv_rep, pres, freq;
  float inv_t;
  float scale;      // GRAD: grad_out * coef
  float lse;        // GRAD
};

template <class T>
__device__ __forceinline__ float sh_to_float(T x);
template <>
__device__ __forceinline__ float sh_to_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float sh_to_float<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <class T>
__device__ __forceinline__ T sh_from_float(float x);
template <>
__device__ __forceinline__ float sh_from_float<float>(float x) { return x; }
// the one rounding of an output to 16 bits (nearest even)
template <>
__device__ __forceinline__ __nv_bfloat16 sh_from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// eight consecutive elements from p; `n` of them exist, `vec`: p is 16-byte aligned
template <class T>
__device__ __forceinline__ void sh_load8(const T* p, int n, bool vec, float* x) {
  if (vec && n == 8) {
    if constexpr (sizeof(T) == 2) {
      const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p));
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    } else {
      const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
      const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
      x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
      x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = j < n ? sh_to_float<T>(p[j]) : 0.f;
  }
}

template <class T>
__device__ __forceinline__ void sh_store8(T* p, int n, bool vec, const float* x) {
  if (vec && n == 8) {
    if constexpr (sizeof(T) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) p[j] = sh_from_float<T>(x[j]);
  }
}

__device__ __forceinline__ bool sh_positive(float x) { return x > 0.f && x < INFINITY; }

// One row's parameters; what points outside its array, or is no valid factor,
// is left out and reported.
template <int MODE>
__device__ __forceinline__ bool sh_load_row(const ShapeArgs& a, int row, ShRow& r, int& bad) {
  const gh_shaping& s = a.s;
  bad = 0;
  bool live = true;
  r.y = -1;
  r.scale = 0.f;
  r.lse = 0.f;
  if (MODE != SHAPE_OUT) {
    live = a.mask[row] != 0;
    r.y = a.targets[row];
  }
  if (MODE == SHAPE_GRAD) {
    const float c = a.coef[row];
    live = live && c != 0.f && a.lse[row] != -INFINITY;  // -inf: the mask leaves nothing, the gradient is 0
    r.scale = (a.grad_out ? *a.grad_out : 1.f) * c;
    r.lse = a.lse[row];
  }
  r.begin = 0;
  r.len = r.plen = 0;
  r.rep = s.repetition ? s.repetition[row] : 1.f;
  r.pres = s.presence ? s.presence[row] : 0.f;
  r.freq = s.frequency ? s.frequency[row] : 0.f;
  float t = s.temperature ? s.temperature[row] : 1.f;
  if (!sh_positive(r.rep)) r.rep = 1.f, bad = 1;
  if (!sh_positive(t)) t = 1.f, bad = 1;
  r.inv_rep = 1.f / r.rep;
  r.inv_t = 1.f / t;
  if (s.hist_len && (r.rep != 1.f || r.pres != 0.f || r.freq != 0.f)) {
    const long long b = s.hist_begin[row];
    const int n = s.hist_len[row];
    if (b < 0 || n < 0 || n > SHAPE_MAX_HIST || b > s.num_tokens - n) {
      bad = 1;
    } else if (n > 0) {
      r.begin = b;
      r.len = n;
      const int p = s.prompt_len ? s.prompt_len[row] : 0;
      r.plen = p < 0 ? 0 : (p < n ? p : n);
    }
  }
  r.bias_b = r.bias_e = 0;
  if (s.bias_set) {
    const int k = s.bias_set[row];
    if (k >= s.num_bias_sets || k < -1) {
      bad = 1;
    } else if (k >= 0) {
      const int b = s.bias_offsets[k], e = s.bias_offsets[k + 1];
      if (b < 0 || e < b || e > s.num_bias || e - b > SHAPE_MAX_BIAS) {
        bad = 1;
      } else if (e > b) {
        r.bias_b = b;
        r.bias_e = e;
      }
    }
  }
  r.allow = -1;
  if (s.allow_row) {
    const int k = s.allow_row[row];
    if (k >= s.num_allow || k < -1)
      bad = 1;
    else
      r.allow = k;
  }
  return live;
}

// Adds history tokens [from, to) of the row that fall into [c0, c0 + cols) to the words.
__device__ __forceinline__ void sh_add_tokens(const int32_t* tokens, const ShRow& r, int from, int to, int c0, int cols,
                                              uint32_t* word, uint32_t* used) {
  const int32_t* h = tokens + r.begin;
#pragma unroll 4
  for (int k = from + threadIdx.x; k < to; k += SH_THREADS) {
    const uint32_t j = static_cast<uint32_t>(h[k] - c0);
    if (j < static_cast<uint32_t>(cols)) {
      if (k < r.plen)
        atomicOr(&word[j], SH_PROMPT);
      else
        atomicAdd(&word[j], 1u);
      atomicOr(&used[j >> 5], 1u << (j & 31));
    }
  }
}

template <class TIn, class TOut, int MODE>
__global__ void __launch_bounds__(SH_THREADS, 3) shape_kernel(const ShapeArgs a) {
  extern __shared__ __align__(16) uint8_t sh_smem[];
  __shared__ ShRow rows[SH_MAX_ROWS];
  __shared__ uint32_t live_bits;
  uint32_t* word = reinterpret_cast<uint32_t*>(sh_smem);
  uint32_t* used = word + (a.table ? a.cols : 0);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile = static_cast<int>(blockIdx.x % a.ntiles);
  const int row0 = static_cast<int>(blockIdx.x / a.ntiles) * a.rows_per_cta;
  const int nrows = min(a.rows_per_cta, a.R - row0);
  const int V = a.V;
  const int c0 = tile * a.cols;
  const int cols = min(a.cols, V - c0);

  if (warp == 0) {
    ShRow r;
    int bad = 0;
    bool live = false;
    if (lane < nrows) live = sh_load_row<MODE>(a, row0 + lane, r, bad);
    if (bad && live && tile == 0) atomicOr(a.status, GH_DEV_BAD_ROW);
    const uint32_t bits = __ballot_sync(0xffffffffu, live);
    const uint32_t before = bits & ((1u << lane) - 1u);
    const int prev = before ? 31 - __clz(before) : 0;
    const long long pb = __shfl_sync(0xffffffffu, r.begin, prev);
    const int pl = __shfl_sync(0xffffffffu, r.len, prev);
    const int pp = __shfl_sync(0xffffffffu, r.plen, prev);
    const int p0 = __shfl_sync(0xffffffffu, r.bias_b, prev);
    const int p1 = __shfl_sync(0xffffffffu, r.bias_e, prev);
    if (live) {
      r.tab = TAB_BUILD;
      r.add_from = 0;
      if (r.len == 0 && r.bias_e == r.bias_b) {
        r.tab = TAB_NONE;
      } else if (before && (pl > 0 || p1 > p0) && p0 == r.bias_b && p1 == r.bias_e && pb == r.begin && pl <= r.len &&
          min(pp, pl) == min(r.plen, pl)) {
        if (pl == r.len) {
          r.tab = TAB_KEEP;
        } else if (pl + 1 == r.len && pl >= r.plen) {
          r.tab = TAB_ADD1;
          r.add_from = a.s.tokens[r.begin + pl];
        } else {
          r.tab = TAB_ADD;
          r.add_from = pl;
        }
      }
      rows[lane] = r;
    }
    if (lane == 0) live_bits = bits;
  }
  __syncthreads();
  const uint32_t bits = live_bits;

  for (int rr = 0; rr < nrows; ++rr) {
    const int row = row0 + rr;
    TOut* out = MODE == SHAPE_LOGP ? nullptr : reinterpret_cast<TOut*>(a.out) + static_cast<size_t>(row) * a.out_ld + c0;
    if (!((bits >> rr) & 1u)) {
      if (MODE == SHAPE_GRAD) {
        const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int j = tid * 8; j < cols; j += SH_THREADS * 8) sh_store8<TOut>(out + j, min(8, cols - j), a.vec_out, zero);
      }
      continue;
    }
    const ShRow& r = rows[rr];
    {
      const int tab = r.tab;
      if (tab == TAB_BUILD) {
        __syncthreads();
        for (int j = tid * 4; j < a.cols; j += SH_THREADS * 4) *reinterpret_cast<uint4*>(word + j) = make_uint4(0, 0, 0, 0);
        for (int j = tid; j < a.cols / 32; j += SH_THREADS) used[j] = 0;
        __syncthreads();
        if (r.bias_e > r.bias_b) {
          for (int k = r.bias_b + tid; k < r.bias_e; k += SH_THREADS) {
            const uint32_t j = static_cast<uint32_t>(a.s.bias_tokens[k] - c0);
            if (j < static_cast<uint32_t>(cols)) {
              // the last entry of a token counts
              atomicMax(&word[j], static_cast<uint32_t>(k - r.bias_b + 1) << SH_BIAS_SHIFT);
              atomicOr(&used[j >> 5], 1u << (j & 31));
            }
          }
          __syncthreads();
        }
        sh_add_tokens(a.s.tokens, r, 0, r.len, c0, cols, word, used);
        __syncthreads();
      } else if (tab == TAB_ADD) {
        __syncthreads();
        sh_add_tokens(a.s.tokens, r, r.add_from, r.len, c0, cols, word, used);
        __syncthreads();
      } else if (tab == TAB_ADD1) {
        const uint32_t j = static_cast<uint32_t>(r.add_from - c0);
        if (j < static_cast<uint32_t>(cols)) {  // the same for every thread: read from shared memory
          __syncthreads();
          if (tid == 0) {
            word[j] += 1u;
            used[j >> 5] |= 1u << (j & 31);
          }
          __syncthreads();
        }
      }
    }

    const TIn* in = reinterpret_cast<const TIn*>(a.logits) + static_cast<size_t>(row) * a.ld + c0;
    const uint8_t* allow =
        r.allow >= 0 ? reinterpret_cast<const uint8_t*>(a.s.allow_bits + static_cast<size_t>(r.allow) * ((V + 31) / 32)) + (c0 >> 3)
                     : nullptr;
    for (int seg = warp * SH_SEG; seg < cols; seg += SH_WARPS * SH_SEG) {
      float x[SH_CHUNKS][8];
      uint32_t ok[SH_CHUNKS];
#pragma unroll
      for (int u = 0; u < SH_CHUNKS; ++u) {
        const int j = seg + u * 256 + lane * 8;
        const int n = min(8, cols - j);
        ok[u] = n <= 0 ? 0u : (n < 8 ? (1u << n) - 1u : 0xffu);
        if (allow && n > 0) ok[u] &= allow[j >> 3];
      }
#pragma unroll
      for (int u = 0; u < SH_CHUNKS; ++u) {
        const int j = seg + u * 256 + lane * 8;
        if (ok[u]) {
          sh_load8<TIn>(in + j, min(8, cols - j), a.vec_in, x[u]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[u][e] = 0.f;
        }
      }
      uint32_t seen[SH_CHUNKS], pos[SH_CHUNKS];  // GRAD: columns whose slope is theta or 1 / theta
#pragma unroll
      for (int u = 0; u < SH_CHUNKS; ++u) {
        const int j = seg + u * 256 + lane * 8;
        seen[u] = pos[u] = 0;
        uint32_t t = 0;
        if (r.tab != TAB_NONE && ok[u]) t = reinterpret_cast<const uint8_t*>(used)[j >> 3] & ok[u];
        if (t) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if ((t >> e) & 1u) {
              const uint32_t w = word[j + e];
              const uint32_t c = w & SH_COUNT;
              float v = x[u][e];
              if (w & (SH_COUNT | SH_PROMPT)) {
                seen[u] |= 1u << e;
                if (v > 0.f) pos[u] |= 1u << e;
                v *= v > 0.f ? r.inv_rep : r.rep;
              }
              v -= r.freq * static_cast<float>(c);
              if (c) v -= r.pres;
              const uint32_t be = w >> SH_BIAS_SHIFT;
              if (be) v += __ldg(a.s.bias_values + r.bias_b + be - 1);
              x[u][e] = v;
            }
          }
        }
      }
      if (MODE == SHAPE_LOGP) {
        float m = -INFINITY;
#pragma unroll
        for (int u = 0; u < SH_CHUNKS; ++u) {
          const int j = seg + u * 256 + lane * 8;
#pragma unroll
          for (int e = 0; e < 8; ++e) x[u][e] = ((ok[u] >> e) & 1u) ? x[u][e] : -INFINITY;
          const int rel = r.y - (c0 + j);
          if (static_cast<uint32_t>(rel) < 8u && r.y < V) {
            float z = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) z = e == rel ? x[u][e] : z;
            a.zy[row] = z * r.inv_t;
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) m = fmaxf(m, x[u][e]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        // the maximum of the raw values is that of the scaled ones; the difference is taken before the step to base
        // 2, where a row of the type's lowest value would overflow
        m *= r.inv_t;
        const float ref = m == -INFINITY ? 0.f : m;
        float sum = 0.f;
#pragma unroll
        for (int u = 0; u < SH_CHUNKS; ++u)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum += ex2_approx(fmaf(x[u][e], r.inv_t, -ref) * SH_LOG2E);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) a.part[static_cast<size_t>(row) * a.nseg + (c0 + seg) / SH_SEG] = make_float2(m, sum);
      } else {
#pragma unroll
        for (int u = 0; u < SH_CHUNKS; ++u) {
          const int j = seg + u * 256 + lane * 8;
          const int n = min(8, cols - j);
          if (n <= 0) continue;
          float o[8];
          if (MODE == SHAPE_OUT) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = ((ok[u] >> e) & 1u) ? x[u][e] * r.inv_t : -INFINITY;
          } else {
            const int rel = r.y - (c0 + j);
            const float g = r.scale * r.inv_t;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float p = ex2_approx(fmaf(x[u][e], r.inv_t, -r.lse) * SH_LOG2E);
              float d = g * ((e == rel ? 1.f : 0.f) - p);
              if ((seen[u] >> e) & 1u) d *= ((pos[u] >> e) & 1u) ? r.inv_rep : r.rep;
              o[e] = ((ok[u] >> e) & 1u) ? d : 0.f;
            }
          }
          sh_store8<TOut>(out + j, n, a.vec_out, o);
        }
      }
    }
  }
}

// A warp per row folds the row's segment partials: lane l takes segments l,
// l + 32, ... in order, then the lanes combine in a xor butterfly.
__global__ void __launch_bounds__(256) shaped_merge_kernel(const ShapeArgs a) {
  const int row = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= a.R) return;
  if (a.mask[row] == 0) {
    if (lane == 0) {
      a.logp[row] = 0.f;
      a.lse_out[row] = 0.f;
    }
    return;
  }
  float m = -INFINITY, s = 0.f;
  const float2* p = a.part + static_cast<size_t>(row) * a.nseg;
  for (int k = lane; k < a.nseg; k += 32) {
    const float2 q = p[k];
    const float mn = fmaxf(m, q.x);
    const float ref = mn == -INFINITY ? 0.f : mn;
    s = s * ex2_approx((m - ref) * SH_LOG2E) + q.y * ex2_approx((q.x - ref) * SH_LOG2E);
    m = mn;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
    const float mn = fmaxf(m, m2);
    const float ref = mn == -INFINITY ? 0.f : mn;
    s = s * ex2_approx((m - ref) * SH_LOG2E) + s2 * ex2_approx((m2 - ref) * SH_LOG2E);
    m = mn;
  }
  if (lane == 0) {
    const int y = a.targets[row];
    const float ls = logf(s);
    const float lse = m + ls;  // -inf when the mask leaves nothing
    float lp;
    if (y >= 0 && y < a.V) {
      const float z = a.zy[row];
      lp = z == -INFINITY ? -INFINITY : (z - m) - ls;
    } else {
      lp = __int_as_float(0x7fc00000);
      atomicOr(a.status, GH_DEV_TARGET_OOR);
    }
    a.logp[row] = lp;
    a.lse_out[row] = lse;
    if (!isfinite(lse) || (y >= 0 && y < a.V && !isfinite(lp))) atomicOr(a.status, GH_DEV_NONFINITE);
  }
}

template <class TIn, class TOut, int MODE>
cudaError_t launch_typed(const ShapeArgs& a, cudaStream_t st) {
  const size_t smem = a.table ? static_cast<size_t>(a.cols) * 4 + a.cols / 8 : 0;
  cudaError_t e = cudaFuncSetAttribute(shape_kernel<TIn, TOut, MODE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       SH_MAX_COLS * 4 + SH_MAX_COLS / 8);
  if (e != cudaSuccess) return e;
  const int64_t blocks = static_cast<int64_t>(a.ntiles) * ceil_div(a.R, a.rows_per_cta);
  shape_kernel<TIn, TOut, MODE><<<static_cast<unsigned>(blocks), SH_THREADS, smem, st>>>(a);
  return cudaGetLastError();
}

template <int MODE>
cudaError_t launch_mode(const ShapeArgs& a, cudaStream_t st) {
  const bool in16 = a.dtype == GH_BF16, out16 = a.out_dtype == GH_BF16;
  if (MODE == SHAPE_OUT) {
    if (in16 != out16)
      return in16 ? launch_typed<__nv_bfloat16, float, SHAPE_OUT>(a, st) : launch_typed<float, __nv_bfloat16, SHAPE_OUT>(a, st);
  }
  return in16 ? launch_typed<__nv_bfloat16, __nv_bfloat16, MODE>(a, st) : launch_typed<float, float, MODE>(a, st);
}

// Columns and rows per CTA.
void plan(ShapeArgs& a) {
  a.cols = SH_MAX_COLS;
  while (a.cols > 4 * SH_SEG && static_cast<int64_t>(a.R) * ceil_div(a.V, a.cols) < 2 * num_sms()) a.cols /= 2;
  a.ntiles = static_cast<int>(ceil_div(a.V, a.cols));
  const int64_t rows = static_cast<int64_t>(a.R) * a.ntiles / (12 * num_sms());
  a.rows_per_cta = static_cast<int>(rows < 1 ? 1 : (rows > SH_MAX_ROWS ? SH_MAX_ROWS : rows));
  a.nseg = static_cast<int>(ceil_div(a.V, SH_SEG));
  a.table = (a.s.hist_len || a.s.bias_set) ? 1 : 0;
  const size_t in_elt = a.dtype == GH_BF16 ? 2 : 4, out_elt = a.out_dtype == GH_BF16 ? 2 : 4;
  a.vec_in = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.ld * in_elt % 16 == 0;
  a.vec_out = reinterpret_cast<uintptr_t>(a.out) % 16 == 0 && a.out_ld * out_elt % 16 == 0;
}

}  // namespace

int64_t shape_segments(int64_t V) { return ceil_div(V, SH_SEG); }

cudaError_t launch_shape(ShapeArgs a, cudaStream_t st) {
  plan(a);
  return launch_mode<SHAPE_OUT>(a, st);
}
cudaError_t launch_shaped_logp(ShapeArgs a, cudaStream_t st) {
  plan(a);
  return launch_mode<SHAPE_LOGP>(a, st);
}
cudaError_t launch_shaped_merge(ShapeArgs a, cudaStream_t st) {
  plan(a);
  shaped_merge_kernel<<<static_cast<unsigned>(ceil_div(a.R, 8)), 256, 0, st>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_shaped_grad(ShapeArgs a, cudaStream_t st) {
  plan(a);
  return launch_mode<SHAPE_GRAD>(a, st);
}

}  // namespace gh
