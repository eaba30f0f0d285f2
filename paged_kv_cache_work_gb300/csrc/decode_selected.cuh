// Attention of each row over a list of its pages (pa_decode_selected): one launch, no workspace.
//
// A unit of work is one new token of one sequence and one kv head with up to 16 of its query
// heads: they share the page list.  The list's 16-token chunks (a page holds a whole number of
// them) are dealt out in tiles to the warps of a thread-block cluster of S CTAs, S chosen from the
// sizes so that few units still spread over the GPU.  Each warp is on its own until the end: it
// looks up 32 chunks of its share at a time (a lane each: list entry, then block table), copies
// its tiles through a private ring of shared-memory stages with 16-byte cp.async (rows that no key
// may be read from are zero-filled, so a masked row never holds NaN or infinity), and keeps its
// own running maximum, sum and accumulator.  No barrier joins the warps while data streams.  At
// the end the warps' states are merged through shared memory, and the CTAs' through distributed
// shared memory, both in a fixed order, by
//     m = max_s m_s, w_s = 2^(m_s - m), l = sum_s w_s l_s, o = sum_s w_s o_s, out = o / l.
//
// Per tile: S = Q K^T on mma.sync m16n8k16 (K fragments by ldmatrix), an online softmax in log2
// units on the accumulators (the running maximum moves only when a logit beats it by 2^8), and
// O += P V with P rounded to the operands' 16-bit type (its sum is kept from the unrounded fp32
// values) and V by ldmatrix.trans.  E4M3 codes become f16 exactly on their way to the MMA; a K
// scale multiplies the logit, a V scale (over the accumulator's own power of two) the weight.
#pragma once

#include <cooperative_groups.h>

#include "decode_mma.cuh"

namespace pa {

struct SelectedParams {
  const char* q;
  const char* k_cache;
  const char* v_cache;
  const float* k_scale;  // null when there is none
  const float* v_scale;
  const int32_t* bt;
  const int32_t* ctx;
  const int32_t* qlens;
  const int32_t* selected;
  const int32_t* num;
  void* out;
  float* lse;
  int32_t* flags;
  long long sc_block;    // scale of (block, slot, head g): block * sc_block + slot * sc_slot +
  int sc_slot, sc_head;  // g * sc_head
  int Sq, Hq, Hkv, G, RB, bs_shift, maxb, nblocks, causal, top_k, split;
  float qk_scale;  // sm_scale * log2(e)
};

// CTAs of a unit's cluster: doubled while the GPU has fewer than two CTAs for each SM and each
// CTA keeps 128 tokens or more.
constexpr int kSelMaxSplit = 8;
inline int selected_split(long long units, long long tokens, int sms) {
  int s = 1;
  while (s < kSelMaxSplit && units * s < 2 * sms && tokens / (2 * s) >= 128) s *= 2;
  return s;
}

template <int D_, int KVK_>
struct SelTraits {
  static constexpr int D = D_;
  static constexpr bool FP8 = KVK_ == KV_FP8;
  static constexpr int BPE = FP8 ? 1 : 2;
  static constexpr int NW = 4;
  static constexpr int NTHREADS = NW * 32;
  static constexpr int ROW = D * BPE;              // bytes of a row
  static constexpr int TK = ROW <= 128 ? 32 : 16;  // tokens of a warp's tile
  static constexpr int SUB = TK / 16;              // 16-token chunks of a tile
  static constexpr int NST = 3;
  static constexpr int TILE = TK * ROW;  // bytes of a K (or V) tile
  static constexpr int SC = FP8 ? 2 * TK * 4 : 0;
  static constexpr int STAGE = 2 * TILE + SC;
  static constexpr int RING = NW * NST * STAGE;
  static constexpr int OSTR = D + 4;  // floats between rows of a staged accumulator
  static constexpr int O_BYTES = 16 * OSTR * 4;
  static constexpr int OFF_ML = round_up(cmax(RING, (NW + 1) * O_BYTES), 128);
  static constexpr int SMEM = OFF_ML + (NW + 1) * 16 * 8;
  static constexpr int CTAS_PER_SM = 2 * (SMEM + 1024) <= 228 * 1024 ? 2 : 1;
  static_assert(SMEM <= 227 * 1024, "shared memory");
};

// 16-byte piece c of row r of a tile: eight rows of a column of pieces lie in distinct banks.
template <class T>
__device__ __forceinline__ uint32_t sel_piece(uint32_t base, int r, int c) {
  const int x = T::ROW >= 128 ? (r & 7) : ((r >> 1) & 3);
  return base + r * T::ROW + ((c ^ x) << 4);
}

__device__ __forceinline__ void cp_async_16_zfill(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_4_zfill(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, int KVK, int QK>
__global__ void __launch_bounds__(SelTraits<D, KVK>::NTHREADS, SelTraits<D, KVK>::CTAS_PER_SM)
    decode_selected_kernel(const SelectedParams p) {
  using T = SelTraits<D, KVK>;
  constexpr bool F16 = T::FP8 || QK == Q_FP16;
  constexpr int KSTEPS = D / 16, NB = D / 8, TK = T::TK, SUB = T::SUB, NT8 = TK / 8;
  extern __shared__ __align__(128) char smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = lane >> 2, qi = lane & 3;
  const int S = p.split, rank = blockIdx.x % S;
  int u = blockIdx.x / S;
  const int rb = u % p.RB;
  u /= p.RB;  // (b * Sq + i) * Hkv + g
  const int g = u % p.Hkv, bi = u / p.Hkv, i = bi % p.Sq, b = bi / p.Sq;
  const uint32_t ring = smem_addr(smem) + warp * T::NST * T::STAGE;
  if constexpr (T::FP8) {
    if (!p.k_scale) {  // no scales: ones that nothing overwrites
      for (int e = lane; e < T::NST * 2 * TK; e += 32)
        *reinterpret_cast<float*>(smem + (warp * T::NST + e / (2 * TK)) * T::STAGE + 2 * T::TILE +
                                  (e % (2 * TK)) * 4) = 1.f;
    }
  }
  grid_dependency_wait();
  grid_dependents_launch();

  // ---- what the row sees, and its list
  const int n = __ldg(p.ctx + b), ql = __ldg(p.qlens + b);
  int L = 0, npages = 0;
  if (ql < 0 || ql > p.Sq || n < ql || (long long)n > ((long long)p.maxb << p.bs_shift)) {
    if (tid == 0 && rank == 0 && i == 0 && g == 0 && rb == 0 && p.flags)
      atomicOr(p.flags, PA_FLAG_BAD_LENGTHS);
  } else if (i < ql) {
    L = p.causal ? n - ql + i + 1 : n;
    npages = (int)(((long long)n + (1 << p.bs_shift) - 1) >> p.bs_shift);
  }
  int count = L > 0 ? __ldg(p.num + u) : 0;
  if (count < 0 || count > p.top_k) {
    if (tid == 0 && rank == 0 && p.flags) atomicOr(p.flags, PA_FLAG_BAD_SELECTION);
    count = count < 0 ? 0 : p.top_k;
  }
  const int cshift = p.bs_shift - 4;  // a page's 16-token chunks
  const long long chunks = (long long)count << cshift;
  const long long tiles = (chunks + SUB - 1) / SUB;
  const long long tile0 = tiles * rank / S, tile1 = tiles * (rank + 1) / S;
  const int my = (int)max(0ll, (tile1 - tile0 - warp + T::NW - 1) / T::NW);  // this warp's tiles
  const int32_t* list = p.selected + (size_t)u * p.top_k;

  // lane l looks up chunk base + l of the warp's chunks (SUB a tile): its block and first token
  int blk = -1, tok = 0, base = -32;
  auto look_up = [&](int x0) {
    base = x0;
    const int x = x0 + lane;
    const long long c = (tile0 + warp + (long long)T::NW * (x / SUB)) * SUB + x % SUB;
    blk = -1;
    if (x / SUB < my && c < chunks) {
      const int page = __ldg(list + (int)(c >> cshift));
      if (page < 0 || page >= npages) {
        if (p.flags) atomicOr(p.flags, PA_FLAG_BAD_SELECTION);
      } else {
        tok = (page << p.bs_shift) + (((int)c & ((1 << cshift) - 1)) << 4);
        blk = __ldg(p.bt + (size_t)b * p.maxb + page);
        if (blk < 0 || blk >= p.nblocks) {
          if (p.flags) atomicOr(p.flags, PA_FLAG_BAD_BLOCK_ID);
          blk = -1;
        }
      }
    }
  };
  // tile j into a stage; valids: for each chunk a byte with its rows that hold visible keys (its
  // first ones)
  uint32_t valid_ring[T::NST];
  auto issue = [&](int j, int stage, uint32_t& valids) {
    valids = 0;
    if (j < my) {
      if (j * SUB >= base + 32) look_up(j * SUB);
      const uint32_t kt = ring + stage * T::STAGE, vt = kt + T::TILE;
      constexpr int PPR = T::ROW / 16;
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        const int x = j * SUB + s - base;
        const int bk = __shfl_sync(kFull, blk, x), t = __shfl_sync(kFull, tok, x);
        const int v = bk < 0 ? 0 : min(max(L - t, 0), 16);
        valids |= (uint32_t)v << (8 * s);
        const int slot = t & ((1 << p.bs_shift) - 1);
        const size_t row0 = v > 0 ? (((size_t)bk << p.bs_shift) + slot) * p.Hkv + g : 0;
        const size_t rstr = (size_t)p.Hkv * T::ROW;
        const char* ks = p.k_cache + row0 * T::ROW;
        const char* vs = p.v_cache + row0 * T::ROW;
#pragma unroll
        for (int e0 = 0; e0 < 16 * PPR; e0 += 32) {
          const int e = e0 + lane, r = e / PPR, c = e % PPR;
          const bool ok = r < v;
          const size_t off = ok ? r * rstr + c * 16 : 0;
          cp_async_16_zfill(sel_piece<T>(kt, s * 16 + r, c), ks + off, ok);
          cp_async_16_zfill(sel_piece<T>(vt, s * 16 + r, c), vs + off, ok);
        }
        if constexpr (T::FP8) {
          if (p.k_scale) {  // lanes 0-15: K scales, lanes 16-31: V scales
            const int r = lane & 15;
            const bool ok = r < v;
            const size_t at = ok ? (size_t)(bk * p.sc_block) + (size_t)((slot + r) * p.sc_slot) +
                                       (size_t)g * p.sc_head
                                 : 0;
            cp_async_4_zfill(kt + 2 * T::TILE + ((lane >> 4) * TK + s * 16 + r) * 4,
                             (lane < 16 ? p.k_scale : p.v_scale) + at, ok);
          }
        }
      }
    }
    cp_async_commit();
  };

  // ---- query fragments: rows quad and quad + 8 are heads rb * 16 + quad (+ 8) of the group.
  // A bf16 row that meets an fp8 cache becomes f16, times the power of two that brings its
  // largest element to [2^7, 2^8): f16's range then holds all that matters of it.
  uint32_t qa[KSTEPS][4];
  float qk_row[2] = {p.qk_scale, p.qk_scale};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int head = rb * 16 + quad + 8 * h;
    const bool real = head < p.G;
    const char* qrow = p.q + (((size_t)bi * p.Hq + (size_t)g * p.G + (real ? head : 0)) * D) * 2;
#pragma unroll
    for (int kk = 0; kk < KSTEPS; ++kk) {
      uint32_t lo = 0, hi = 0;
      if (real) {
        if constexpr (T::FP8) {  // permuted k order: channels 16 kk + 4 qi + {0, 1}, {2, 3}
          const uint2 v = __ldg(reinterpret_cast<const uint2*>(qrow + (16 * kk + 4 * qi) * 2));
          lo = v.x;
          hi = v.y;
        } else {
          lo = __ldg(reinterpret_cast<const uint32_t*>(qrow + (16 * kk + 2 * qi) * 2));
          hi = __ldg(reinterpret_cast<const uint32_t*>(qrow + (16 * kk + 8 + 2 * qi) * 2));
        }
      }
      qa[kk][h] = lo;
      qa[kk][2 + h] = hi;
    }
    if constexpr (T::FP8 && QK == Q_BF16) {
      float big = 0.f;
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk) {
        const float2 a = bf16x2_to_f2(qa[kk][h]), c = bf16x2_to_f2(qa[kk][2 + h]);
        big = fmaxf(big, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(c.x), fabsf(c.y))));
      }
      big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
      big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
      const float up = fmaxf(pow2_above(big), 0x1p-100f);  // (mul stays finite)
      const float mul = pow2_inverse(up) * 256.f;
      qk_row[h] *= up * (1.f / 256.f);
#pragma unroll
      for (int kk = 0; kk < KSTEPS; ++kk) {
        const float2 a = bf16x2_to_f2(qa[kk][h]), c = bf16x2_to_f2(qa[kk][2 + h]);
        qa[kk][h] = pack2<true>(a.x * mul, a.y * mul);
        qa[kk][2 + h] = pack2<true>(c.x * mul, c.y * mul);
      }
    }
  }

  float o[NB][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) o[nb][0] = o[nb][1] = o[nb][2] = o[nb][3] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
  float vref = kPow2Least, vinv = pow2_inverse(kPow2Least) * kPLift;  // fp8: o is in units of vref / kPLift

  if (my > 0) look_up(0);
  __syncwarp();
#pragma unroll
  for (int s = 0; s < T::NST - 1; ++s) issue(s, s, valid_ring[s]);
  const int mat = lane >> 3;
  for (int j0 = 0; j0 < my; j0 += T::NST) {
#pragma unroll
    for (int st = 0; st < T::NST; ++st) {
      const int j = j0 + st;
      if (j >= my) break;
      cp_async_wait_group<T::NST - 2>();
      __syncwarp();
      constexpr int last = T::NST - 1;
      issue(j + last, (st + last) % T::NST, valid_ring[(st + last) % T::NST]);
      const uint32_t valids = valid_ring[st];
      const uint32_t kt = ring + st * T::STAGE, vt = kt + T::TILE;
      const float* sks = reinterpret_cast<const float*>(smem + (warp * T::NST + st) * T::STAGE + 2 * T::TILE);
      const float* svs = sks + TK;

      // ---- S = Q K^T
      float sacc[NT8][4];
#pragma unroll
      for (int nb = 0; nb < NT8; ++nb) sacc[nb][0] = sacc[nb][1] = sacc[nb][2] = sacc[nb][3] = 0.f;
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        if constexpr (!T::FP8) {
          const int row = s * 16 + (lane & 7) + ((mat >> 1) << 3);
#pragma unroll
          for (int kk = 0; kk < KSTEPS; ++kk) {
            uint32_t r0, r1, r2, r3;
            ldsm_x4(sel_piece<T>(kt, row, 2 * kk + (mat & 1)), r0, r1, r2, r3);
            mma16816<F16>(sacc[2 * s], qa[kk], r0, r1);
            mma16816<F16>(sacc[2 * s + 1], qa[kk], r2, r3);
          }
        } else {
          const int row = s * 16 + (lane & 7) + ((mat & 1) << 3);
#pragma unroll
          for (int kk = 0; kk < KSTEPS; kk += 2) {
            uint32_t r[4];
            ldsm_x4(sel_piece<T>(kt, row, kk + (mat >> 1)), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int nb = 0; nb < 2; ++nb) {
                const uint32_t w4 = r[2 * h + nb];
                mma16816<true>(sacc[2 * s + nb], qa[kk + h], e4m3x2_to_f16x2(w4),
                               e4m3x2_to_f16x2(w4 >> 16));
              }
          }
        }
      }

      // ---- online softmax: sacc[nb] holds tokens 8 nb + 2 qi + {0, 1} of rows quad, quad + 8
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nb = 0; nb < NT8; ++nb) {
        const int v = (valids >> (8 * (nb >> 1))) & 255;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = (nb & 1) * 8 + 2 * qi + (e & 1);
          float x = sacc[nb][e] * qk_row[e >> 1];
          if constexpr (T::FP8) x *= sks[8 * nb + 2 * qi + (e & 1)];
          x = t < v ? x : -INFINITY;
          sacc[nb][e] = x;
          mx[e >> 1] = fmaxf(mx[e >> 1], x);
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(kFull, mx[h], 2));
      }
      const bool need0 = mx[0] > m_run[0] + 8.f, need1 = mx[1] > m_run[1] + 8.f;
      if (__any_sync(kFull, need0 || need1)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float mn = (h ? need1 : need0) ? mx[h] : m_run[h];
          const float alpha = mn == m_run[h] ? 1.f : fast_exp2(m_run[h] - mn);
          m_run[h] = mn;
          l_run[h] *= alpha;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            o[nb][2 * h] *= alpha;
            o[nb][2 * h + 1] *= alpha;
          }
        }
      }
      if constexpr (T::FP8) {
        // magnitudes order as their bits do; rows that may not be read hold zeros
        const float big = __uint_as_float(
            __reduce_max_sync(kFull, __float_as_uint(fabsf(svs[lane & (TK - 1)]))));
        if (big > vref) {  // warp-uniform
          const float up = pow2_above(big), f = vref * pow2_inverse(up);
          vref = up;
          vinv = pow2_inverse(up) * kPLift;
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nb][e] *= f;
        }
      }
      uint32_t pa[SUB][4];
#pragma unroll
      for (int nb = 0; nb < NT8; ++nb) {
        float pr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = sacc[nb][e];
          pr[e] = x != -INFINITY ? fast_exp2(x - m_run[e >> 1]) : 0.f;
          l_run[e >> 1] += pr[e];
          if constexpr (T::FP8) pr[e] *= svs[8 * nb + 2 * qi + (e & 1)] * vinv;
        }
        pa[nb >> 1][2 * (nb & 1)] = pack2<F16>(pr[0], pr[1]);
        pa[nb >> 1][2 * (nb & 1) + 1] = pack2<F16>(pr[2], pr[3]);
      }

      // ---- O += P V
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        const int row = s * 16 + (lane & 7) + ((mat & 1) << 3);
        if constexpr (!T::FP8) {
#pragma unroll
          for (int nd = 0; nd < KSTEPS; ++nd) {
            uint32_t r0, r1, r2, r3;
            ldsm_x4_t(sel_piece<T>(vt, row, 2 * nd + (mat >> 1)), r0, r1, r2, r3);
            mma16816<F16>(o[2 * nd], pa[s], r0, r1);
            mma16816<F16>(o[2 * nd + 1], pa[s], r2, r3);
          }
        } else {
          // a transposed pair holds tokens (2 qi, 2 qi + 1) of channels (2 quad, 2 quad + 1):
          // n-block 2 c gets the even channels of 16-channel chunk c, 2 c + 1 the odd ones
#pragma unroll
          for (int c2 = 0; c2 < KSTEPS; c2 += 2) {
            uint32_t r[4];
            ldsm_x4_t(sel_piece<T>(vt, row, c2 + (mat >> 1)), r[0], r[1], r[2], r[3]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t lo = r[2 * h], hi = r[2 * h + 1];
              mma16816<true>(o[2 * (c2 + h)], pa[s], e4m3x2_to_f16x2(prmt(lo, 0, 0x0020)),
                             e4m3x2_to_f16x2(prmt(hi, 0, 0x0020)));
              mma16816<true>(o[2 * (c2 + h) + 1], pa[s], e4m3x2_to_f16x2(prmt(lo, 0, 0x0031)),
                             e4m3x2_to_f16x2(prmt(hi, 0, 0x0031)));
            }
          }
        }
      }
    }
  }
  cp_async_wait_all();
  if constexpr (T::FP8) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[nb][e] *= vref * (1.f / kPLift);
  }

  // ---- merge the warps
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l_run[h] += __shfl_xor_sync(kFull, l_run[h], 1);
    l_run[h] += __shfl_xor_sync(kFull, l_run[h], 2);
  }
  float* const obuf = reinterpret_cast<float*>(smem);  // [NW + 1][16][OSTR]; the last: merged
  float2* const ml = reinterpret_cast<float2*>(smem + T::OFF_ML);  // [NW + 1][16] (max, sum)
  __syncthreads();  // every warp is done with its stages
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float* row = obuf + (warp * 16 + quad + 8 * h) * T::OSTR;
#pragma unroll
    for (int c = 0; c < KSTEPS; ++c) {
      if constexpr (T::FP8) {
        *reinterpret_cast<float4*>(row + 16 * c + 4 * qi) =
            make_float4(o[2 * c][2 * h], o[2 * c + 1][2 * h], o[2 * c][2 * h + 1], o[2 * c + 1][2 * h + 1]);
      } else {
        *reinterpret_cast<float2*>(row + 16 * c + 2 * qi) = make_float2(o[2 * c][2 * h], o[2 * c][2 * h + 1]);
        *reinterpret_cast<float2*>(row + 16 * c + 8 + 2 * qi) =
            make_float2(o[2 * c + 1][2 * h], o[2 * c + 1][2 * h + 1]);
      }
    }
    if (qi == 0) ml[warp * 16 + quad + 8 * h] = make_float2(m_run[h], l_run[h]);
  }
  __syncthreads();

  constexpr int D4 = D / 4;
  const int rows = min(16, p.G - rb * 16);
  // states s = 0 .. states - 1 of a row merged: (max, sum) at ml_of(s), accumulator at o_of(s)
  auto merge = [&](int r, int d4, int states, auto ml_of, auto o_of, float4& O, float2& st) {
    float m = -INFINITY;
    for (int s = 0; s < states; ++s) m = fmaxf(m, ml_of(s)->x);
    float l = 0.f;
    O = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s = 0; s < states; ++s) {
      const float2 x = *ml_of(s);
      if (x.y == 0.f) continue;  // no key in this state
      const float w = fast_exp2(x.x - m);
      const float4 v = *reinterpret_cast<const float4*>(o_of(s) + r * T::OSTR + 4 * d4);
      l = __fmaf_rn(w, x.y, l);
      O.x = __fmaf_rn(w, v.x, O.x);
      O.y = __fmaf_rn(w, v.y, O.y);
      O.z = __fmaf_rn(w, v.z, O.z);
      O.w = __fmaf_rn(w, v.w, O.w);
    }
    st = make_float2(m, l);
  };
  auto finish = [&](int r, int d4, const float4& O, const float2& st) {
    const float inv = st.y == 0.f ? 0.f : 1.f / st.y;  // no key: zero (NaN stays NaN)
    const size_t row = (size_t)bi * p.Hq + (size_t)g * p.G + rb * 16 + r;
    store_out4<QK>(p.out, row * D + 4 * d4, make_float4(O.x * inv, O.y * inv, O.z * inv, O.w * inv));
    if (d4 == 0 && p.lse) p.lse[row] = st.y == 0.f ? -INFINITY : (st.x + fast_log2(st.y)) * kLn2;
  };
  for (int e = tid; e < rows * D4; e += T::NTHREADS) {
    const int r = e / D4, d4 = e % D4;
    float4 O;
    float2 st;
    merge(r, d4, T::NW, [&](int s) { return ml + s * 16 + r; },
          [&](int s) { return obuf + s * 16 * T::OSTR; }, O, st);
    if (S == 1) {
      finish(r, d4, O, st);
    } else {
      *reinterpret_cast<float4*>(obuf + (T::NW * 16 + r) * T::OSTR + 4 * d4) = O;
      if (d4 == 0) ml[T::NW * 16 + r] = st;
    }
  }
  if (S == 1) return;

  // ---- merge the cluster's CTAs: each finishes its share of the rows' pieces
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  for (int e = rank * T::NTHREADS + tid; e < rows * D4; e += S * T::NTHREADS) {
    const int r = e / D4, d4 = e % D4;
    float4 O;
    float2 st;
    merge(r, d4, S, [&](int s) { return cluster.map_shared_rank(ml + T::NW * 16 + r, s); },
          [&](int s) { return cluster.map_shared_rank(obuf + T::NW * 16 * T::OSTR, s); }, O, st);
    finish(r, d4, O, st);
  }
  cluster.sync();  // nobody leaves while its shared memory is read
}

template <int D, int KVK, int QK>
cudaError_t launch_selected(const SelectedParams& p, long long units, cudaStream_t s) {
  using T = SelTraits<D, KVK>;
  auto kern = decode_selected_kernel<D, KVK, QK>;
  static std::atomic<uint64_t> attr_done{0};  // devices whose limit is raised
  const cudaError_t e = set_smem_attr_once(attr_done, reinterpret_cast<const void*>(kern), T::SMEM);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * p.split));
  cfg.blockDim = dim3(T::NTHREADS);
  cfg.dynamicSmemBytes = T::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int D>
cudaError_t launch_selected_for_dim(const SelectedParams& p, int kvk, int qk, long long units,
                                    cudaStream_t s) {
  if (kvk == KV_FP8)
    return qk == Q_BF16 ? launch_selected<D, KV_FP8, Q_BF16>(p, units, s)
                        : launch_selected<D, KV_FP8, Q_FP16>(p, units, s);
  return qk == Q_BF16 ? launch_selected<D, KV_BF16, Q_BF16>(p, units, s)
                      : launch_selected<D, KV_FP16, Q_FP16>(p, units, s);
}

cudaError_t launch_selected_d64(const SelectedParams& p, int kvk, int qk, long long units, cudaStream_t s);
cudaError_t launch_selected_d128(const SelectedParams& p, int kvk, int qk, long long units, cudaStream_t s);
cudaError_t launch_selected_d256(const SelectedParams& p, int kvk, int qk, long long units, cudaStream_t s);

}  // namespace pa
