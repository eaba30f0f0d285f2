// K and V rows into their places in the cache, as pa_append_kv and pa_append_rotated write them: D / 8
// lanes a row, eight consecutive elements (16 bytes of input) a lane, one to four rows a warp.
#pragma once

#include <type_traits>

#include "append_block.cuh"
#include "int4.cuh"

namespace pa {

// What a cache holds of a row.
enum StoreKind { STORE_16 = 0, STORE_FP8 = 1, STORE_INT4 = 2 };

inline int store_kind(const pa_config& c) {
  return c.kv_dtype == PA_INT4 ? STORE_INT4 : c.kv_dtype == PA_FP8_E4M3 ? STORE_FP8 : STORE_16;
}

// How queries and keys are made ready on their way (pa_rotary; half = 0: no rotation).
struct RotateParams {
  const char* q_weight;
  const char* k_weight;
  const float* cos_sin;
  const int32_t* positions;
  int half, interleaved, table_rows, axes, axis1, axis2;  // pairs from axis1 (axis2) on: next axis
  float eps;
};

struct AppendParams {
  const char* q;
  const char* k_new;
  const char* v_new;
  const int32_t* bt;
  const int32_t* ctx;
  const int32_t* qlens;
  char* q_out;
  char* k_out;
  char* k_cache;
  char* v_cache;
  void* k_scale;
  void* v_scale;
  int32_t* flags;
  long long q_stride, k_stride, v_stride;  // elements between tokens
  int tokens;                              // B * Sq
  int Sq, Hq, Hkv, bs, bs_shift, maxb, nblocks, scale_mode;
  int q_steps, k_steps, v_steps;  // steps of a token's q, k and v rows (none where none are wanted)
  int parts, per;    // they are the work of `parts` warps, `per` steps each
  FastDiv part_div, token_div;  // by parts and by Sq
  RotateParams r;
};

// Head dims 64, 128 and 256, in append.cu (no rotation) and rotate.cu.
cudaError_t launch_append(const AppendParams& p, int head_dim, int qk, int kind, cudaStream_t s);
cudaError_t launch_rotate(const AppendParams& p, int head_dim, int qk, int kind, cudaStream_t s);

// Splits a token's rows over warps: as many steps a warp as leave 32 warps an SM (at most 24: the steps
// share the token's lengths, positions and angles), at least two past 24 warps an SM (what is resident of
// most instances at once), the same for each of the token's warps.  A step is one to four rows of one kind.
// Tokens behind a sequence's last count as the others do: their number is only known on the GPU.
//   Measured: 32 sequences of 4 tokens, 16 kv heads of 256 (4,096 steps), fp8 per token 2.8 us (3.9 with one
// step a warp, a part of them in a second wave), 4 bits 3.3 (4.2), 16 bits 2.2 (2.45); rotating 32 of 8,
// 32 heads on 8 of 128, 4.0 (5.6).  4 prompts of 2,048 such fp8 rows 57 us in 16 and 16 steps of a token's
// 32, 75 in 24 and 8.  As many steps as all warps are resident with: 4 chunks of 512, 32 heads on 4, 8.6 us
// in place of 7.4.
inline void split_rows(AppendParams& p, int head_dim, int sms, bool stores) {
  const int rows_per_step = 256 / head_dim;
  p.q_steps = ceil_div(p.Hq, rows_per_step);
  p.k_steps = ceil_div(p.Hkv, rows_per_step);
  p.v_steps = stores ? p.k_steps : 0;
  const int steps = p.q_steps + p.k_steps + p.v_steps;
  const long long all = (long long)p.tokens * steps, spare = all / ((long long)sms * 32);
  const int least = all > (long long)sms * 24 ? 2 : 1;
  p.parts = ceil_div(steps, (int)(spare < least ? least : spare > 24 ? 24 : spare));
  p.per = ceil_div(steps, p.parts);
  p.part_div = FastDiv((uint32_t)p.parts);
  p.token_div = FastDiv((uint32_t)p.Sq);
}

#if defined(__CUDACC__)

template <int QK>
__device__ __forceinline__ void widen_row(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = pair_values<QK>(u[k]);
    x[2 * k] = f.x;
    x[2 * k + 1] = f.y;
  }
}
template <int QK>
__device__ __forceinline__ uint4 narrow_row(const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (QK == Q_BF16) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
      u[k] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      const __half2 h = __floats2half2_rn(x[2 * k], x[2 * k + 1]);
      u[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Eight E4M3 codes of the lane's elements in one of the scale modes of a token, a tensor or none;
// the row's scale in *scale_of_row.
template <int L>
__device__ __forceinline__ uint2 codes_fp8(const float (&x)[8], const float* scale, int scale_mode,
                                           float* scale_of_row) {
  uint32_t c[4];
  if (scale_mode == PA_SCALE_NONE) {
#pragma unroll
    for (int k = 0; k < 4; ++k) c[k] = e4m3x2_rn_sat(x[2 * k], x[2 * k + 1]);
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  }
  float y[8], s;
  if (scale_mode == PA_SCALE_PER_TOKEN) {
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fabsf(y[k] = x[k]));
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, o));
    s = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
    *scale_of_row = s;
  } else {
    s = __ldg(scale);
    const float top = s * 512.f;  // (past it a quotient by a plain scale saturates all the same)
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] = fabsf(x[k]) > top ? copysignf(top, x[k]) : x[k];
  }
  if (s >= 0x1p-60f && s <= 0x1p60f) {
    // IEEE quotients by one step from the rounded reciprocal (a y below 2^-70 gives a code of zero by
    // either way).  With eight IEEE divisions in their place an append of one row with a tensor's scale
    // took 3.2 us in place of 2.2, 8 prompts of 2,048 rows of 8 heads of 128 33.6 in place of 30.1.
    const float inv = __fdiv_rn(1.f, s);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      c[k] = e4m3x2_rn_sat(quotient(y[2 * k], s, inv), quotient(y[2 * k + 1], s, inv));
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      c[k] = e4m3x2_rn_sat(__fdiv_rn(x[2 * k], s), __fdiv_rn(x[2 * k + 1], s));
  }
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// The row over the root of its mean square, times the weight.  The whole warp is here.
template <int QK, int L>
__device__ __forceinline__ void normalise(float (&x)[8], const uint4& weight, float eps) {
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) sum = __fmaf_rn(x[e], x[e], sum);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  const float inv = rsqrtf(__fmaf_rn(sum, 1.f / (8 * L), eps));
  float f[8];
  widen_row<QK>(weight, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * f[e];
}

// A warp takes up to 24 steps of one token's rows, q's before k's before v's, each a row (or two, four)
// of one kind; loops by kind keep what only queries or keys need out of the others' instructions.
//   Measured (replayed): rotating append of 8 prompts of up to 4,096 tokens, 32 heads on 8 of 128, three
// axes, 16-bit cache (405 MB) 83.7 us, 4.8 TB/s, bound by instructions (0.53 of a slot a cycle; 130 us
// with steps of mixed kinds and eight a warp); one token of 32 sequences 2.8 us; 8 chunks of up to 512
// rows into a 4-bit cache, 8 heads of 128, about 10 us, most of it the chain of a row's minimum, maximum,
// step and quotients.  Three CTAs an SM: two take 102 us, four (64 registers) 88.
template <int D, int QK, int KIND, bool ROT>
__global__ void __launch_bounds__(256, KIND == STORE_16 && !ROT ? 4 : 3) append_kernel(const AppendParams p) {
  constexpr int L = D / 8, RPS = 32 / L;  // lanes of a row, rows of a step
  constexpr int U = 4;                    // steps whose rows are loaded together
  const int lane = threadIdx.x & 31, sub = lane / L, c0 = lane % L * 8;
  const long long warps = (long long)gridDim.x * 8, all = (long long)p.tokens * p.parts;
  const int k_step = ROT ? p.q_steps : 0, v_step = k_step + p.k_steps, steps = v_step + p.v_steps;
  grid_dependency_wait();
  for (long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); w < all; w += warps) {
    int token, part;
    if (all <= INT32_MAX) {
      token = (int)p.part_div.div((uint32_t)w);
      part = (int)w - token * p.parts;
    } else {
      token = (int)(w / p.parts);
      part = (int)(w % p.parts);
    }
    const int b = (int)p.token_div.div((uint32_t)token), i = token - b * p.Sq;
    const int n = __ldg(p.ctx + b), ql = __ldg(p.qlens + b);
    const long long cap = (long long)p.maxb << p.bs_shift;
    if (ql < 0 || ql > p.Sq || n < ql || (long long)n > cap) {
      if (lane == 0 && i == 0 && part == 0 && p.flags) atomicOr(p.flags, PA_FLAG_BAD_LENGTHS);
      continue;
    }
    if (i >= ql) continue;
    const int pos = n - ql + i, first = part * p.per, end = min(steps, first + p.per);
    // the token's angles: of channels c0 .. c0 + 7 (interleaved: of their four pairs); the sine is
    // negative where the pair's other channel is subtracted
    float cs[8], sn[8];
    bool turns = false, all_turn = false;
    if constexpr (ROT) {
      if (p.r.half > 0) {
        int at[3] = {pos, pos, pos};
        bool bad = false;
#pragma unroll
        for (int a = 0; a < 3; ++a) {
          if (a >= p.r.axes) break;
          if (p.r.positions) at[a] = __ldg(p.r.positions + (size_t)a * p.tokens + token);
          bad |= at[a] < 0 || at[a] >= p.r.table_rows;
        }
        if (bad) {
          if (lane == 0 && p.flags) atomicOr(p.flags, PA_FLAG_BAD_POSITION);
          continue;
        }
        all_turn = 2 * p.r.half == D;
        turns = c0 < 2 * p.r.half;
        const bool second = c0 >= p.r.half;  // (of half-split pairs)
        const int pair = p.r.interleaved ? c0 / 2 : second ? c0 - p.r.half : c0;
        if (turns && first < v_step) {
          auto axis = [&](int x) { return x < p.r.axis1 ? at[0] : x < p.r.axis2 ? at[1] : at[2]; };
#pragma unroll
          for (int e = 0; e < 8; e += 4) {
            if (e == 4 && p.r.interleaved) break;
            const int x = pair + e, lo = axis(x), hi = axis(x + 3);
            const float* row = p.r.cos_sin + (size_t)lo * (2 * p.r.half) + x;
            if (p.r.axes == 1 || (lo == hi && axis(x + 1) == lo && axis(x + 2) == lo)) {
              const float4 c = __ldg(reinterpret_cast<const float4*>(row));
              const float4 s = __ldg(reinterpret_cast<const float4*>(row + p.r.half));
              cs[e] = c.x, cs[e + 1] = c.y, cs[e + 2] = c.z, cs[e + 3] = c.w;
              sn[e] = s.x, sn[e + 1] = s.y, sn[e + 2] = s.z, sn[e + 3] = s.w;
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float* y = p.r.cos_sin + (size_t)axis(x + k) * (2 * p.r.half) + x + k;
                cs[e + k] = __ldg(y);
                sn[e + k] = __ldg(y + p.r.half);
              }
            }
          }
          if (!p.r.interleaved && !second) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sn[e] = -sn[e];
          }
        }
      }
    }
    int blk = -1;
    if (p.k_cache && end > k_step) {
      blk = __ldg(p.bt + (size_t)b * p.maxb + (pos >> p.bs_shift));
      if (blk < 0 || blk >= p.nblocks) {
        if (lane == 0 && p.flags) atomicOr(p.flags, PA_FLAG_BAD_BLOCK_ID);
        blk = -1;
      }
    }
    uint4 wq = make_uint4(0, 0, 0, 0), wk = wq;
    if constexpr (ROT) {
      if (p.r.q_weight) wq = __ldg(reinterpret_cast<const uint4*>(p.r.q_weight) + lane % L);
      if (p.r.k_weight) wk = __ldg(reinterpret_cast<const uint4*>(p.r.k_weight) + lane % L);
    }
    const int slot = pos & (p.bs - 1);
    const size_t crow0 = ((size_t)max(blk, 0) * p.bs + slot) * p.Hkv;
    // steps [s0, s1) of the rows of one kind, `rows` of them, from `src` on
    enum { ROW_Q, ROW_K, ROW_V };
    auto run = [&](auto kind_, int s0, int s1, int rows, const char* src, char* dense, char* cache,
                   void* scale) {
      constexpr int ROWS = decltype(kind_)::value;
      int h = s0 * RPS + sub;
      src += (size_t)h * (D * 2) + c0 * 2;
      dense += (size_t)h * (D * 2) + c0 * 2;
      const uint4 weight = ROWS == ROW_Q ? wq : wk;
      const bool norm = ROT && ROWS != ROW_V && (ROWS == ROW_Q ? p.r.q_weight : p.r.k_weight) != nullptr;
      const bool writes = ROT && (ROWS == ROW_Q || (ROWS == ROW_K && p.k_out));
      for (; s0 < s1; s0 += U, h += U * RPS, src += U * RPS * D * 2, dense += U * RPS * D * 2) {
        uint4 in[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {  // (in place: a row is read here and written below, by the same lanes)
          in[k] = make_uint4(0, 0, 0, 0);
          if (s0 + k < s1 && h + k * RPS < rows) in[k] = *reinterpret_cast<const uint4*>(src + k * RPS * D * 2);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          if (s0 + k >= s1) break;
          const int g = h + k * RPS;
          const bool real = g < rows;
          uint4 out = in[k];
          float x[8];
          if ((ROT && ROWS != ROW_V) || KIND != STORE_16) widen_row<QK>(in[k], x);
          if constexpr (ROT && ROWS != ROW_V) {
            if (norm) normalise<QK, L>(x, weight, p.r.eps);
            if (p.r.half > 0) {
              float y[8];  // the row turned
              if (p.r.interleaved) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                  y[e] = x[e] * cs[e / 2] - x[e + 1] * sn[e / 2];
                  y[e + 1] = x[e + 1] * cs[e / 2] + x[e] * sn[e / 2];
                }
              } else {
                const int away = p.r.half / 8;  // lanes to the pair's other channel
                const int from = !turns ? lane : c0 >= p.r.half ? lane - away : lane + away;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                  y[e] = __fmaf_rn(__shfl_sync(kFull, x[e], from), sn[e], x[e] * cs[e]);
              }
              if (all_turn) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = y[e];
              } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = turns ? y[e] : x[e];
              }
            }
            out = narrow_row<QK>(x);
            if (real && writes) *reinterpret_cast<uint4*>(dense + k * RPS * D * 2) = out;
          }
          if constexpr (ROWS != ROW_Q) {
            if (!p.k_cache) continue;
            const bool stores = real && blk >= 0;
            const size_t crow = crow0 + (stores ? g : 0);
            if constexpr (KIND == STORE_16) {
              if (stores) *reinterpret_cast<uint4*>(cache + (crow * D + c0) * 2) = out;
            } else if constexpr (KIND == STORE_FP8) {
              float s;
              const uint2 c = codes_fp8<L>(x, static_cast<const float*>(scale), p.scale_mode, &s);
              if (stores) {
                *reinterpret_cast<uint2*>(cache + crow * D + c0) = c;
                if (c0 == 0 && p.scale_mode == PA_SCALE_PER_TOKEN) static_cast<float*>(scale)[crow] = s;
              }
            } else {
              uint32_t pair;
              const uint32_t c = quantise_row<QK, L>(x, &pair);
              if (stores) {
                *reinterpret_cast<uint32_t*>(cache + (crow * D + c0) / 2) = c;
                if (c0 == 0)
                  static_cast<uint32_t*>(scale)[((size_t)blk * p.Hkv + g) * p.bs + slot] = pair;
              }
            }
          }
        }
      }
    };
    if (ROT && first < k_step)
      run(std::integral_constant<int, ROW_Q>(), first, min(end, k_step), p.Hq,
          p.q + (size_t)token * p.q_stride * 2, p.q_out + (size_t)token * p.Hq * (D * 2), nullptr, nullptr);
    if (first < v_step && end > k_step)
      run(std::integral_constant<int, ROW_K>(), max(first - k_step, 0), min(end, v_step) - k_step, p.Hkv,
          p.k_new + (size_t)token * p.k_stride * 2, p.k_out + (size_t)token * p.Hkv * (D * 2), p.k_cache,
          p.k_scale);
    if (end > v_step)
      run(std::integral_constant<int, ROW_V>(), max(first - v_step, 0), end - v_step, p.Hkv,
          p.v_new + (size_t)token * p.v_stride * 2, nullptr, p.v_cache, p.v_scale);
  }
  grid_dependents_launch();
}

template <int D, bool ROT>
cudaError_t launch_append_d(const AppendParams& p, int qk, int kind, cudaStream_t s) {
  const long long ctas = ((long long)p.tokens * p.parts + 7) / 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(ctas < (1 << 30) ? ctas : 1 << 30));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
#define PA_APPEND(KIND_)                                                                      \
  if (kind == KIND_)                                                                          \
    return qk == Q_BF16 ? cudaLaunchKernelEx(&cfg, append_kernel<D, Q_BF16, KIND_, ROT>, p)   \
                        : cudaLaunchKernelEx(&cfg, append_kernel<D, Q_FP16, KIND_, ROT>, p);
  PA_APPEND(STORE_16)
  PA_APPEND(STORE_FP8)
  PA_APPEND(STORE_INT4)
#undef PA_APPEND
  return cudaErrorNotSupported;
}

#endif  // __CUDACC__

}  // namespace pa
