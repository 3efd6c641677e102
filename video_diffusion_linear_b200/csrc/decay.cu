// Linear attention with a decay for each head: the fp32 scan, the states before the segments, the
// single-token step, and the C entry points.
#include <cmath>

#include "check.h"
#include "common.cuh"
#include "decay.h"
#include "internal.h"

namespace vdn {

// ---------------------------------------------------------------- fp32 scan
// S_t = lambda S_{t-1} + z_t y_t^T, o_t = S_t x_t token by token, the state in registers: a thread
// owns R rows x CC columns of one (batch, head, segment), `unit`.  Per token and thread R CC
// multiplies and 2 R CC multiply-adds in packed pairs, against CC / 2 vector loads of x and y that
// all rows share (a vector load takes four cycles of the SM's one load path however few addresses it has:
// 8 x 16 spends 160 cycles on loads and 384 on arithmetic per token, 2 x 64 512 on loads).  The chunked form has no
// fewer operations here: its products with the state cost the same 4 d^2 per token, and without tensor cores the near
// terms come on top.  Few rows leave an SM one unit of four warps, so a token's chain of loads, multiply-adds and
// shuffles bounds it: 0.28 us per token with its output, 0.18 without (d = 128).  The gradients of 2 x 777 tokens x 4
// heads (five launches of up to 128 blocks and two prefixes): 114 us, 14 us of them arithmetic at the fp32 rate (5 %
// more with tiles of 4 tokens, a barrier each; 14 % with one token at a time).
namespace {

template <int D> struct ScanShape;
template <> struct ScanShape<128> {
  static constexpr int R = 8, CC = 16, kUnits = 1, kTok = 8, kStages = 4, kUnroll = 2;
};
template <> struct ScanShape<16> {
  static constexpr int R = 2, CC = 4, kUnits = 2, kTok = 8, kStages = 8, kUnroll = 4;
};

__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// N tokens of a tile from token k0 on: their loads, and their sums over the parts, overlap.  first: the decay into the
// first of them; out: the first one's output of this thread's row, step elements apart.
template <int D, bool kOut, int N, int kArrays>
__device__ __forceinline__ void scan_tokens(float2 (&s)[ScanShape<D>::R][ScanShape<D>::CC / 2],
                                            const float (&tk)[kArrays][ScanShape<D>::kTok][D], int k0, float first,
                                            float lambda, float add, int row0, int part, float* out, long long step,
                                            float out_scale) {
  constexpr int R = ScanShape<D>::R, CC = ScanShape<D>::CC, kParts = D / CC;
  float4 yv[N][CC / 4];
  float zv[N][R];
#pragma unroll
  for (int j = 0; j < N; ++j) {
#pragma unroll
    for (int i = 0; i < CC / 4; ++i) yv[j][i] = *reinterpret_cast<const float4*>(&tk[0][k0 + j][4 * (kParts * i + part)]);
    static_assert(R == 2 || R % 4 == 0, "vector loads of z");
    if constexpr (R == 2) {
      const float2 f = *reinterpret_cast<const float2*>(&tk[1][k0 + j][row0]);
      zv[j][0] = f.x * add;
      zv[j][1] = f.y * add;
    } else {
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const float4 f = *reinterpret_cast<const float4*>(&tk[1][k0 + j][row0 + r]);
        zv[j][r] = f.x * add; zv[j][r + 1] = f.y * add; zv[j][r + 2] = f.z * add; zv[j][r + 3] = f.w * add;
      }
    }
  }
  float o[N][R];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float l = j == 0 ? first : lambda;
    float2 acc[R][2];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r][0] = acc[r][1] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < CC / 4; ++i) {
      float4 xv;
      if (kOut) xv = *reinterpret_cast<const float4*>(&tk[kArrays - 1][k0 + j][4 * (kParts * i + part)]);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2 zr = make_float2(zv[j][r], zv[j][r]);
        float2& a = s[r][2 * i];
        float2& c = s[r][2 * i + 1];
        a = __ffma2_rn(zr, make_float2(yv[j][i].x, yv[j][i].y), __fmul2_rn(a, make_float2(l, l)));
        c = __ffma2_rn(zr, make_float2(yv[j][i].z, yv[j][i].w), __fmul2_rn(c, make_float2(l, l)));
        if (kOut) {
          acc[r][0] = __ffma2_rn(a, make_float2(xv.x, xv.y), acc[r][0]);
          acc[r][1] = __ffma2_rn(c, make_float2(xv.z, xv.w), acc[r][1]);
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) o[j][r] = (acc[r][0].x + acc[r][0].y) + (acc[r][1].x + acc[r][1].y);
  }
  if constexpr (kOut) {
    // the parts' sums of R rows: whole rows while there are more parts than rows, then each step halves the rows
    // that a thread holds, until one is left
#pragma unroll
    for (int w = kParts / 2; w >= R; w >>= 1)
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) o[j][r] += __shfl_xor_sync(0xffffffffu, o[j][r], w);
#pragma unroll
    for (int w = R / 2; w > 0; w >>= 1) {
      const bool up = part & w;
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int r = 0; r < w; ++r) {
          const float give = up ? o[j][r] : o[j][r + w], keep = up ? o[j][r + w] : o[j][r];
          o[j][r] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
    }
    static_assert(kParts >= R && (D / R) * kParts % 32 == 0, "whole warps reduce");
    if (part < R)
#pragma unroll
      for (int j = 0; j < N; ++j)
        out[j * step] = o[j][0] * out_scale;
  }
}

// kOut: the scan (reads x, writes o and the final state); else a segment's own state
template <int D, bool kRev, bool kOut>
__global__ void __launch_bounds__(ScanShape<D>::kUnits * (D / ScanShape<D>::R) * (D / ScanShape<D>::CC))
    k_decay_scan(const float* __restrict__ x, const float* __restrict__ y, const float* __restrict__ z, int B, int H,
                 int T, int nseg, int seg_len, const float* __restrict__ decay, const int* __restrict__ lengths,
                 const float* init, const float* __restrict__ seg_states, int transposed, float out_scale, float add, int clear,
                 float* __restrict__ out, float* final, float* __restrict__ states, uint32_t* __restrict__ status, int clear_status) {
  using Sh = ScanShape<D>;
  constexpr int R = Sh::R, CC = Sh::CC, kParts = D / CC, kTok = Sh::kTok;
  constexpr int kUnitThreads = (D / R) * kParts, kArrays = kOut ? 3 : 2, kVec = D / 4;
  constexpr int kStages = Sh::kStages;
  __shared__ __align__(16) float tile[kStages][Sh::kUnits][kArrays][kTok][D];   // y, z, x
  const long long BH = (long long)B * H, units = BH * (kOut ? nseg : nseg - 1);
  const int tid = threadIdx.x, u = tid / kUnitThreads, ut = tid % kUnitThreads;
  if (clear_status && blockIdx.x == 0 && tid == 0) *status = 0;
  const long long unit = (long long)blockIdx.x * Sh::kUnits + u;
  const bool live = unit < units;
  const long long bh = live ? unit % BH : 0;
  // a segment's own state: nothing follows the order's last segment
  const int seg = live ? (int)(unit / BH) + (!kOut && kRev ? 1 : 0) : 0, h = (int)(bh % H), b = (int)(bh / H);
  const int n_tok = decay_tokens(lengths, b, T), t0 = seg * seg_len;
  const int t1 = live ? min(n_tok, t0 + seg_len) : 0;
  const int n = max(0, t1 - t0);
  int n_max = n;                                         // tokens of the block's longest unit
  for (int o = 0; o < Sh::kUnits; ++o) {
    const long long other = (long long)blockIdx.x * Sh::kUnits + o;
    if (other < units) {
      const int ot0 = ((int)(other / BH) + (!kOut && kRev ? 1 : 0)) * seg_len;
      n_max = max(n_max, min(decay_tokens(lengths, (int)(other % BH / H), T), ot0 + seg_len) - ot0);
    }
  }
  const float lambda = decay_factor(decay[h]);
  const int part = ut % kParts, row0 = ut / kParts * R;   // rows row0 .. row0 + R - 1, float4 columns kParts i + part

  float2 s[R][CC / 2];
  const float* src = !kOut ? nullptr : nseg > 1 ? seg_states + unit * D * D : init ? init + bh * D * D : nullptr;
#pragma unroll
  for (int i = 0; i < CC / 4; ++i) {
    const int col = 4 * (kParts * i + part);
#pragma unroll
    for (int r = 0; r < R; ++r) s[r][2 * i] = s[r][2 * i + 1] = make_float2(0.f, 0.f);
    if (live && src) {
      if (!transposed) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 f = *reinterpret_cast<const float4*>(src + (row0 + r) * D + col);
          s[r][2 * i] = make_float2(f.x, f.y);
          s[r][2 * i + 1] = make_float2(f.z, f.w);
        }
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          s[r][2 * i] = make_float2(src[col * D + row0 + r], src[(col + 1) * D + row0 + r]);
          s[r][2 * i + 1] = make_float2(src[(col + 2) * D + row0 + r], src[(col + 3) * D + row0 + r]);
        }
      }
    }
  }

  // token k of the scan order
  auto token = [&](int k) { return kRev ? t1 - 1 - k : t0 + k; };
  auto load = [&](int tl, int buf) {
    for (int e = ut; e < kArrays * kTok * kVec; e += kUnitThreads) {
      const int c = e % kVec, k = e / kVec % kTok, a = e / (kVec * kTok), at = tl * kTok + k;
      if (at < n) {
        const float* g = a == 0 ? y : a == 1 ? z : x;
        cp_async16(&tile[buf][u][a][k][4 * c], g + (((long long)b * T + token(at)) * H + h) * D + 4 * c);
      }
    }
    cp_async_commit();
  };
  const int tiles = (n_max + kTok - 1) / kTok;
  // kStages - 1 tiles ahead; a group is committed for every tile, loaded or not, so that the count tells the tile
  for (int tl = 0; tl < kStages - 1; ++tl) {
    if (tl < tiles) load(tl, tl);
    else cp_async_commit();
  }
  for (int tl = 0; tl < tiles; ++tl) {
    cp_async_wait<kStages - 2>();
    __syncthreads();                            // tile tl is there, and everyone is done with tile tl - 1
    if (tl + kStages - 1 < tiles) load(tl + kStages - 1, (tl + kStages - 1) % kStages);
    else cp_async_commit();
    const int buf = tl % kStages;
    const int kn = min(kTok, n - tl * kTok);
    const long long step = (kRev ? -1 : 1) * (long long)H * D;
    float* o = kOut ? out + (((long long)b * T + token(tl * kTok)) * H + h) * D + row0 + part : nullptr;
    // reverse: the state enters the first token undecayed
    float first = kRev && tl == 0 && !isnan(lambda) ? 1.f : lambda;
    int k = 0;
    for (; k + Sh::kUnroll <= kn; k += Sh::kUnroll, first = lambda)
      scan_tokens<D, kOut, Sh::kUnroll>(s, tile[buf][u], k, first, lambda, add, row0, part, o + k * step, step, out_scale);
    for (; k < kn; ++k, first = lambda)
      scan_tokens<D, kOut, 1>(s, tile[buf][u], k, first, lambda, add, row0, part, o + k * step, step, out_scale);
  }
  cp_async_wait<0>();
  if (!live) return;
  if (kOut && clear) {                          // rows of the segment behind the sequence
    const int c0 = max(t0, t1), c1 = min(T, t0 + seg_len);
    for (int i = ut; i < (c1 - c0) * D; i += kUnitThreads) out[(((long long)b * T + c0 + i / D) * H + h) * D + i % D] = 0.f;
  }
  const int last_seg = kRev || n_tok == 0 ? 0 : (n_tok - 1) / seg_len;
  float* dst = kOut ? (final && seg == last_seg ? final + bh * D * D : nullptr) : n > 0 ? states + (seg * BH + bh) * D * D : nullptr;
  if (!dst) return;
  const float l_end = kRev && n > 0 ? lambda : 1.f;
#pragma unroll
  for (int i = 0; i < CC / 4; ++i) {
    const int col = 4 * (kParts * i + part);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const float4 f = make_float4(s[r][2 * i].x * l_end, s[r][2 * i].y * l_end, s[r][2 * i + 1].x * l_end,
                                   s[r][2 * i + 1].y * l_end);
      if (kOut && transposed) {
        dst[col * D + row0 + r] = f.x;
        dst[(col + 1) * D + row0 + r] = f.y;
        dst[(col + 2) * D + row0 + r] = f.z;
        dst[(col + 3) * D + row0 + r] = f.w;
      } else {
        *reinterpret_cast<float4*>(dst + (row0 + r) * D + col) = f;
      }
    }
  }
}

template <int D, bool kOut> cudaError_t launch_scan(const DecayScan& s, const DecayPlan& p, float* states) {
  using Sh = ScanShape<D>;
  const long long units = (long long)s.B * s.H * (kOut ? p.nseg : p.nseg - 1);
  const unsigned grid = (unsigned)((units + Sh::kUnits - 1) / Sh::kUnits);
  const int threads = Sh::kUnits * (D / Sh::R) * (D / Sh::CC);
  auto kern = s.reverse ? k_decay_scan<D, true, kOut> : k_decay_scan<D, false, kOut>;
  kern<<<grid, threads, 0, s.stream>>>((const float*)s.x, (const float*)s.y, (const float*)s.z, s.B, s.H, s.T, p.nseg,
                                       p.len, s.decay, s.lengths, s.init, s.seg_states, s.transposed ? 1 : 0,
                                       s.out_near, s.add, s.clear ? 1 : 0, (float*)s.out, s.final, states, s.status, s.clear_status ? 1 : 0);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_segments_simt(const DecayScan& s, const DecayPlan& p, float* states) {
  return s.d == 16 ? launch_scan<16, false>(s, p, states) : launch_scan<128, false>(s, p, states);
}
cudaError_t launch_decay_scan_simt(const DecayScan& s, const DecayPlan& p) {
  return s.d == 16 ? launch_scan<16, true>(s, p, nullptr) : launch_scan<128, true>(s, p, nullptr);
}

// ---------------------------------------------------------------- states before the segments
// In scan order: out_s = in, in <- lambda^{tokens of s} in + own_s.  One thread per four state entries.  Bound by
// the latency of the loads, so eight segments' own states are read at once, ahead of the stores over them.
namespace {

constexpr int kPrefixBatch = 8;

__global__ void __launch_bounds__(128) k_decay_prefix(int B, int H, int T, int d, int nseg, int seg_len,
                                                      const float* __restrict__ decay, const int* __restrict__ lengths,
                                                      const float* __restrict__ init, int reverse, float* states) {
  const int vecs = d * d / 4;
  const long long BH = (long long)B * H, i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= BH * vecs) return;
  const long long bh = i / vecs;
  const int n_tok = decay_tokens(lengths, (int)(bh / H), T);
  const float l2 = decay_log2(decay[bh % H]);
  float4 run = init ? reinterpret_cast<const float4*>(init)[i] : make_float4(0.f, 0.f, 0.f, 0.f);
  float4* st = reinterpret_cast<float4*>(states) + i;
  auto segment = [&](int k) { return reverse ? nseg - 1 - k : k; };
  auto tokens = [&](int k) { return min(n_tok - segment(k) * seg_len, seg_len); };
  for (int k0 = 0; k0 < nseg; k0 += kPrefixBatch) {
    float4 own[kPrefixBatch];
#pragma unroll
    for (int j = 0; j < kPrefixBatch; ++j)      // none of the order's last segment, nor of one without tokens
      own[j] = k0 + j + 1 < nseg && tokens(k0 + j) > 0 ? st[segment(k0 + j) * BH * vecs] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kPrefixBatch; ++j) {
      const int k = k0 + j, n = tokens(k);
      if (k >= nseg) break;
      st[segment(k) * BH * vecs] = run;
      if (n > 0) {
        const float w = exp2f((float)n * l2);
        run = make_float4(fmaf(w, run.x, own[j].x), fmaf(w, run.y, own[j].y), fmaf(w, run.z, own[j].z),
                          fmaf(w, run.w, own[j].w));
      }
    }
  }
}

}  // namespace

cudaError_t launch_decay_prefix(const DecayScan& s, const DecayPlan& p, float* states) {
  const long long n = (long long)s.B * s.H * s.d * s.d / 4;
  k_decay_prefix<<<(unsigned)((n + 127) / 128), 128, 0, s.stream>>>(s.B, s.H, s.T, s.d, p.nseg, p.len, s.decay,
                                                                    s.lengths, s.init, s.reverse ? 1 : 0, states);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- single token
// One pass over the state: S <- lambda S + v k^T, o = scale S q.  Bound by the state's bytes (2 x 64 KB
// per row and head at d = 128).  A warp takes eight rows, a row per load instruction (512 bytes), all
// eight loads in flight before the first use; a (row of the batch, head) is split over four CTAs so that
// a single sequence still reaches most SMs.  256 rows x 24 heads: 132 us, 6.1 TB/s, bf16 and fp32 alike; one row x 24
// heads: 6 us with a cold L2, below the 10 us that the binding takes to issue it.
//
// With slots, the state of row b lies in slot slots[b].  The CTA of the first row that names a slot
// takes every later row of that slot too, in row order: they are steps of one sequence.  Every CTA looks through all
// slots for that (B / 128 loads a thread: nothing against its 8 KB of state, but for thousands of rows with small states).
namespace {

constexpr int kStepThreads = 128;

template <int D, typename T>
__global__ void __launch_bounds__(kStepThreads)
    k_decay_step(int B, int H, const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v,
                 const float* __restrict__ decay, float* __restrict__ state, const int* __restrict__ slots,
                 int n_slots, float scale, T* __restrict__ out) {
  constexpr int kRowLanes = D / 4;                 // lanes of one state row
  constexpr int kWarpRows = 32 / kRowLanes;        // rows of one load instruction of a warp
  constexpr int kLoads = D == 128 ? 8 : 2;
  constexpr int kRows = kWarpRows * kLoads;        // rows per warp
  constexpr int kWarpsPerHead = D / kRows;         // 16 (d = 128) or 1 (d = 16)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_row = (H * kWarpsPerHead + 3) / 4;                   // CTAs of one row of the batch
  const int b = blockIdx.x / per_row, wi = (blockIdx.x % per_row) * 4 + warp;
  const int h = wi / kWarpsPerHead;
  const bool live = h < H;
  const int slot = slots ? slots[b] : b;
  if (slot < 0 || slot >= n_slots) return;         // the whole CTA: no sequence in this row
  const int row0 = (wi % kWarpsPerHead) * kRows + lane / kRowLanes, c4 = lane % kRowLanes;
  float4* st = reinterpret_cast<float4*>(state + (((long long)slot * H + h) * D + row0) * D) + c4;
  float4 s[kLoads];
  if (live)
#pragma unroll
    for (int i = 0; i < kLoads; ++i) s[i] = st[i * kWarpRows * kRowLanes];
  bool again = false;
  if (slots) {
    bool early = false, late = false;
    for (int o = threadIdx.x; o < B; o += kStepThreads)
      if (slots[o] == slot) {
        early |= o < b;
        late |= o > b;
      }
    if (__syncthreads_or(early)) return;           // an earlier row's CTA takes this one
    again = __syncthreads_or(late);
  }
  if (!live) return;
  const float lambda = decay_factor(decay[h]);
  for (int row = b;;) {
    const long long at = ((long long)row * H + h) * D;
    float kv[4], qv[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      kv[e] = to_f32(k[at + 4 * c4 + e]);
      qv[e] = to_f32(q[at + 4 * c4 + e]);
    }
    float o[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const float vr = to_f32(v[at + row0 + i * kWarpRows]);
      s[i].x = fmaf(lambda, s[i].x, vr * kv[0]);
      s[i].y = fmaf(lambda, s[i].y, vr * kv[1]);
      s[i].z = fmaf(lambda, s[i].z, vr * kv[2]);
      s[i].w = fmaf(lambda, s[i].w, vr * kv[3]);
      o[i] = fmaf(s[i].x, qv[0], s[i].y * qv[1]) + fmaf(s[i].z, qv[2], s[i].w * qv[3]);
    }
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
      for (int w = kRowLanes / 2; w > 0; w >>= 1) o[i] += __shfl_xor_sync(0xffffffffu, o[i], w);
    if (c4 == 0)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) out[at + row0 + i * kWarpRows] = from_f32<T>(o[i] * scale);
    if (!again) break;
    do ++row;
    while (row < B && slots[row] != slot);
    if (row >= B) break;
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) st[i * kWarpRows * kRowLanes] = s[i];
}

}  // namespace

cudaError_t launch_decay_step(const vdn_shape& sh, const void* q, const void* k, const void* v, const float* decay,
                              float* state, const int* slots, int n_slots, float scale, void* out,
                              cudaStream_t stream) {
  const int warps = sh.d == 128 ? 16 : 1;
  const unsigned grid = (unsigned)((long long)sh.B * ((sh.H * warps + 3) / 4));
#define VDN_STEP(D_, T_)                                                                                        \
  k_decay_step<D_, T_><<<grid, kStepThreads, 0, stream>>>(sh.B, sh.H, (const T_*)q, (const T_*)k, (const T_*)v, \
                                                          decay, state, slots, n_slots, scale, (T_*)out)
  if (sh.dtype == VDN_DTYPE_BF16) VDN_STEP(128, __nv_bfloat16);
  else if (sh.d == 128) VDN_STEP(128, float);
  else VDN_STEP(16, float);
#undef VDN_STEP
  return cudaGetLastError();
}

// ---------------------------------------------------------------- plan
// Into how many segments the token axis is split.  One segment per (batch, head) needs no second pass over k and
// v; more fill the SMs when there are few rows.  The choice is the smallest estimate of
//   waves(rows) (start + units scan)                                    (one segment)
//   waves(rows nseg) (2 start + units / nseg (scan + own)) + rest       (split: own states, prefix, scan)
// with measured times per unit (a chunk of 128 tokens, or a token) and per block, for the forward; the gradients take
// the same segments.  A split pays from 1024 tokens on the tensor-core path with two heads (20 us against 36 us), and
// above 148 rows too where the last wave of one pass would be poorly filled.  There, split against one pass, forward
// and gradients in us: fp32 160 rows of 2048 tokens 1120 against 1324 and 2890 against 3945; bf16 150 rows of 20000
// 1030 against 1070 and 2610 against 2880, but 150 rows of 8192 459 against 435 and 1169 against 1154.  It goes by the
// padded length: the lengths are on the device.  fp32, d = 128: two blocks fit an SM, the estimate counts one.
struct DecayCost {
  int unit, least, slots;          // tokens per unit, units per segment at least, segments that run at once
  double start, scan, own, rest;   // microseconds
};
static DecayCost decay_cost(const vdn_shape& sh) {
  if (use_tc(sh, VDN_IMPL_AUTO)) return {kDecayChunk, 2, 148, 4.0, 3.5, 1.7, 9.0};
  return sh.d == 128 ? DecayCost{1, 32, 148, 3.0, 0.28, 0.18, 9.0}
                     : DecayCost{1, 32, 148 * 8, 3.0, 0.11, 0.07, 9.0};
}

DecayPlan plan_decay(const vdn_shape& sh, bool backward) {
  static const int kSplits[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 40, 48, 64, 80, 96, 128, 148};
  const DecayCost c = decay_cost(sh);
  const long long T = (long long)sh.F * sh.S, BH = (long long)sh.B * sh.H, units = (T + c.unit - 1) / c.unit;
  DecayPlan p;
  long long per_best = units;
  double best = 0.0;
  for (int nseg : kSplits) {
    const long long per = (units + nseg - 1) / nseg;
    if (nseg > 1 && per < c.least) break;
    const double waves = (double)((BH * ((units + per - 1) / per) + c.slots - 1) / c.slots);
    const double cost = nseg == 1 ? waves * (c.start + per * c.scan)
                                  : waves * (2 * c.start + per * (c.scan + c.own)) + c.rest;
    if (nseg == 1 || cost < best) {
      best = cost;
      per_best = per;
    }
  }
  p.nseg = (int)((units + per_best - 1) / per_best);
  p.len = (int)(per_best * c.unit);
  size_t off = 256;
  if (p.nseg > 1) {
    const size_t bytes = (size_t)p.nseg * BH * sh.d * sh.d * sizeof(float);
    p.states = off;
    off += bytes;
    if (backward) {
      p.rstates = off;
      off += bytes;
    }
  }
  p.total = (off + 255) & ~(size_t)255;
  return p;
}

}  // namespace vdn

// ---------------------------------------------------------------- C entry points
using namespace vdn;

namespace {

vdn_status decay_shape(const vdn_shape* sh) {
  const vdn_status s = check_shape(sh);
  if (s != VDN_OK) return s;
  // grids of (batch, head, segment) and of (batch, quarter of a head); token indices with a segment added stay in int32
  if ((long long)sh->B * sh->H > (1 << 24) || (long long)sh->F * sh->S > (1 << 30)) return VDN_ERR_UNSUPPORTED;
  return VDN_OK;
}

// bf16 has no form of the scan without the tensor cores (the fp32 kernels would read its buffers as floats)
vdn_status scan_shape(const vdn_shape* sh) {
  const vdn_status s = decay_shape(sh);
  return s == VDN_OK && sh->dtype == VDN_DTYPE_BF16 && !use_tc(*sh, VDN_IMPL_AUTO) ? VDN_ERR_UNSUPPORTED : s;
}

cudaError_t run_scan(const DecayScan& s, const DecayPlan& p, bool tc) {
  return tc ? launch_decay_scan_tc(s, p) : launch_decay_scan_simt(s, p);
}
// the states before the segments of scan `s`, into `states`
cudaError_t run_segments(const DecayScan& s, const DecayPlan& p, bool tc, float* states) {
  const cudaError_t e = tc ? launch_decay_segments_tc(s, p, states) : launch_decay_segments_simt(s, p, states);
  return e != cudaSuccess ? e : launch_decay_prefix(s, p, states);
}

}  // namespace

extern "C" {

size_t vdn_decay_workspace_size(const vdn_shape* shape) {
  return scan_shape(shape) == VDN_OK ? plan_decay(*shape, false).total : 0;
}
size_t vdn_decay_backward_workspace_size(const vdn_shape* shape) {
  return scan_shape(shape) == VDN_OK ? plan_decay(*shape, true).total : 0;
}

vdn_status vdn_decay_forward(const vdn_shape* shape, const void* q, const void* k, const void* v, const float* decay,
                             const float* state_in, const int* lengths, int clear, float scale, void* workspace,
                             size_t workspace_bytes, void* out, float* state_out, void* stream) {
  vdn_status st = scan_shape(shape);
  if (st != VDN_OK) return st;
  if (!q || !k || !v || !decay || !workspace || !out || !std::isfinite(scale) || (clear != 0 && clear != 1))
    return VDN_ERR_INVALID_ARG;
  const vdn_shape& sh = *shape;
  const DecayPlan p = plan_decay(sh, false);
  const size_t big = token_bytes(sh), sb = (size_t)sh.B * sh.H * sh.d * sh.d * sizeof(float);
  Buffers buf;
  buf.in(q, big);
  buf.in(k, big);
  buf.in(v, big);
  buf.in(decay, (size_t)sh.H * 4);
  // a state may be carried in place: state_out == state_in
  if (state_in != state_out) buf.in(state_in, sb);
  buf.in(lengths, (size_t)sh.B * 4);
  buf.out(out, big);
  buf.out(state_out, sb);
  buf.workspace(workspace, p.total);
  if ((st = buf.check()) != VDN_OK) return st;
  if (workspace_bytes < p.total) return VDN_ERR_WORKSPACE;

  const bool tc = use_tc(sh, VDN_IMPL_AUTO);
  const float sc = scale > 0.f ? scale : 1.0f / std::sqrt((float)sh.d);
  char* ws = static_cast<char*>(workspace);
  DecayScan s{};
  s.B = sh.B; s.H = sh.H; s.T = sh.F * sh.S; s.d = sh.d;
  s.x = q; s.y = k; s.z = v;
  s.decay = decay; s.lengths = lengths;
  s.init = state_in;
  s.out_near = s.out_far = sc;
  s.add = 1.f;
  s.exact_state = true;   // taken or not: out does not depend on it
  s.clear = clear && lengths;
  s.out = out; s.final = state_out;
  s.status = reinterpret_cast<uint32_t*>(ws + p.status);
  s.stream = (cudaStream_t)stream;
  s.clear_status = true;
  cudaError_t e = cudaSuccess;
  if (p.nseg > 1) {
    float* states = reinterpret_cast<float*>(ws + p.states);
    e = run_segments(s, p, tc, states);
    s.seg_states = states;
    s.clear_status = false;
  }
  if (e == cudaSuccess) e = run_scan(s, p, tc);
  return e == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
}

vdn_status vdn_decay_backward(const vdn_shape* shape, const void* q, const void* k, const void* v, const float* decay,
                              const float* state_in, const int* lengths, int clear, float scale, const void* dout,
                              const float* dstate_out, void* workspace, size_t workspace_bytes, void* dq, void* dk,
                              void* dv, float* dstate_in, void* stream) {
  vdn_status st = scan_shape(shape);
  if (st != VDN_OK) return st;
  if (!q || !k || !v || !decay || !dout || !workspace || !dq || !dk || !dv || !std::isfinite(scale) ||
      (clear != 0 && clear != 1))
    return VDN_ERR_INVALID_ARG;
  const vdn_shape& sh = *shape;
  const DecayPlan p = plan_decay(sh, true);
  const size_t big = token_bytes(sh), sb = (size_t)sh.B * sh.H * sh.d * sh.d * sizeof(float);
  Buffers buf;
  buf.in(q, big);
  buf.in(k, big);
  buf.in(v, big);
  buf.in(dout, big);
  buf.in(decay, (size_t)sh.H * 4);
  buf.in(state_in, sb);
  buf.in(dstate_out, sb);
  buf.in(lengths, (size_t)sh.B * 4);
  buf.out(dq, big);
  buf.out(dk, big);
  buf.out(dv, big);
  buf.out(dstate_in, sb);
  buf.workspace(workspace, p.total);
  if ((st = buf.check()) != VDN_OK) return st;
  if (workspace_bytes < p.total) return VDN_ERR_WORKSPACE;

  const bool tc = use_tc(sh, VDN_IMPL_AUTO);
  const float sc = scale > 0.f ? scale : 1.0f / std::sqrt((float)sh.d);
  char* ws = static_cast<char*>(workspace);
  // The state's gradient is kept to fp32 rounding where the call has a state, whether its gradient is taken or not, so
  // that dv and dk do not depend on that.  A call without a state pays for it only when it asks for the gradient
  // (48360 tokens x 24 heads: 1080 us, else 1000).
  const bool exact = state_in != nullptr || dstate_in != nullptr;
  float *fs = nullptr, *rs = nullptr;
  DecayScan s{};
  s.B = sh.B; s.H = sh.H; s.T = sh.F * sh.S; s.d = sh.d;
  s.decay = decay; s.lengths = lengths;
  s.clear = clear && lengths;
  s.status = reinterpret_cast<uint32_t*>(ws + p.status);
  s.stream = (cudaStream_t)stream;
  s.clear_status = true;
  cudaError_t e = cudaSuccess;
  if (p.nseg > 1) {
    fs = reinterpret_cast<float*>(ws + p.states);
    rs = reinterpret_cast<float*>(ws + p.rstates);
    DecayScan f = s;                      // the states before the segments: sum lambda^.. v k^T
    f.y = k; f.z = v; f.init = state_in; f.add = 1.f;
    e = run_segments(f, p, tc, fs);
    s.clear_status = false;
    DecayScan r = s;                      // their gradients from the end: scale sum lambda^.. do q^T
    r.y = q; r.z = dout; r.init = dstate_out; r.add = sc; r.reverse = true;
    r.exact_state = exact;
    if (e == cudaSuccess) e = run_segments(r, p, tc, rs);
  }
  // dq_i = scale S_i^T do_i: the scan of z = k, y = v, whose state is S^T, read by do
  DecayScan a = s;
  a.x = dout; a.y = v; a.z = k;
  a.init = state_in; a.seg_states = fs; a.transposed = true;
  a.out_near = a.out_far = sc; a.add = 1.f;
  a.out = dq;
  if (e == cudaSuccess) e = run_scan(a, p, tc);
  s.clear_status = false;
  // R_j = dL/dS_j = lambda R_{j+1} + scale do_j q_j^T:  dk_j = R_j^T v_j,  dv_j = R_j k_j
  DecayScan c = s;
  c.reverse = true;
  c.init = dstate_out; c.seg_states = rs;
  c.out_near = tc ? sc : 1.f; c.out_far = 1.f; c.add = sc;
  DecayScan dks = c;
  dks.x = v; dks.y = dout; dks.z = q; dks.transposed = true; dks.out = dk;
  if (e == cudaSuccess) e = run_scan(dks, p, tc);
  c.x = k; c.y = q; c.z = dout; c.out = dv; c.final = dstate_in;
  c.exact_state = exact;
  if (e == cudaSuccess) e = run_scan(c, p, tc);
  return e == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
}

vdn_status vdn_decay_step(const vdn_shape* shape, const void* q, const void* k, const void* v, const float* decay,
                          float* state, const int* slots, int n_slots, float scale, void* out, void* stream) {
  vdn_status st = decay_shape(shape);
  if (st != VDN_OK) return st;
  const vdn_shape& sh = *shape;
  if (sh.F != 1 || sh.S != 1) return VDN_ERR_INVALID_ARG;
  if (!q || !k || !v || !decay || !state || !out || n_slots < 1 || !std::isfinite(scale)) return VDN_ERR_INVALID_ARG;
  if (!slots && n_slots != sh.B) return VDN_ERR_INVALID_ARG;
  const size_t big = token_bytes(sh);
  Buffers buf;
  buf.in(q, big);
  buf.in(k, big);
  buf.in(v, big);
  buf.in(decay, (size_t)sh.H * 4);
  buf.in(slots, (size_t)sh.B * 4);
  buf.out(out, big);
  buf.out(state, (size_t)n_slots * sh.H * sh.d * sh.d * sizeof(float));
  if ((st = buf.check()) != VDN_OK) return st;
  const float sc = scale > 0.f ? scale : 1.0f / std::sqrt((float)sh.d);
  return launch_decay_step(sh, q, k, v, decay, state, slots, n_slots, sc, out, (cudaStream_t)stream) == cudaSuccess
             ? VDN_OK
             : VDN_ERR_CUDA;
}

}  // extern "C"
