// Linear attention with a decay for each head, on the tensor cores (bf16, d = 128).
//
//   S_t = lambda S_{t-1} + z_t y_t^T,  o_t = S_t x_t
// in chunks of C = 128 tokens.  With i, j the token's place in the chunk and S the state at its start:
//   P_ij = lambda^{i-j} (x_i . y_j), j <= i            X Y^T
//   o_i  = sum_j P_ij z_j + lambda^{i+1} S x_i         P Z and X S^T
//   S   <- lambda^n S + sum_j z_j (lambda^{n-1-j} y_j)^T      Z^T Yd
// (from the last token to the first: P_ij = lambda^{j-i}, j >= i; the state's factor is lambda^{n-1-i}
// and a token's factor lambda^{j+1}).  All exponents are >= 0, so no power leaves the fp32 range.
//
// Precision.  The state stays in fp32 (registers) and every sum in fp32 (TMEM).  The decayed keys
// Yd are products of a bf16 and an fp32 number, and their product runs on bf16 operands: as three bf16
// terms they are good to 2^-23 and the state is an fp32 quantity, which it is where the state can leave the call
// (DecayScan::exact_state); where it only feeds bf16 outputs, two terms (2^-15) are as good and a third cheaper.
// Two operands are rounded to bf16 once, 2^-8 of their size at most, as the output itself is: P, and
// the state as it enters X S^T.
//
// P and the decayed keys (as Yd^T, transposed on the way by ldmatrix) are A operands in TMEM, which spares
// writing them to shared memory: that is what the elementwise warps, the copies and the products share.  The
// state's product is formed transposed for it (lane = y channel).  An MMA of 128 x 128 x 16 takes 64 cycles here
// with A in either place, 90 - 100 while the other units work too.
//
// Bound by the chain of dependent steps within a chunk, not by one unit: X Y^T -> weights -> P Z -> output on one
// side, keys -> their product -> state -> X S^T on the other, about 6000 cycles per chunk, products 39 - 47 % of
// them and DRAM at 52 - 57 % of its rate: 59 - 61 us for 12288 tokens x 24 heads; all of a call, 48360 tokens: forward
// 400 - 430 us, gradients (five passes) 940 - 1020, by the clock that the power cap leaves.  What counts besides is the code of a chunk, which the warps' roles fetch from
// different places: loops that are not unrolled and one instance of each step brought 72 us (three terms) and 67
// (reverse) to 60 and 59.  What was tried and is slower: fewer, fuller warps (4 + 8), waits that suspend the thread
// (+ 2.5 %) or are called, the state's part decayed by the state's warps, both halves of a row loaded at once (spills).
#include <atomic>

#include "common.cuh"
#include "decay.h"
#include "tc.cuh"
#include "tmap.h"

namespace vdn {

namespace {

constexpr int kC = kDecayChunk;
constexpr uint32_t kTile = 32768;          // 128 tokens x 128 channels bf16, SW128: two halves of 64 channels
constexpr int kNearWarps = 8, kStateWarps = 16;
constexpr int kTmaWarp = kNearWarps + kStateWarps, kMmaWarp = kTmaWarp + 1, kStoreWarp = kTmaWarp + 2;
constexpr int kThreads = 32 * (kStoreWarp + 1);
constexpr uint32_t kIdescKK = tc::idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t kIdescKM = tc::idesc_bf16_f32(128, 128, false, true);

// byte offset of the 16-byte chunk c (0..15) of row r in a tile
__device__ __forceinline__ uint32_t tile_chunk(int r, int c) {
  return (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// The factors lambda^{...} times the scan's `add` of a chunk's tokens, two tokens to a word, as three bf16 terms
// (2^-24 of them is left).
struct KeyTable {
  uint32_t w[3][kC / 2];
};
// entry of tokens 2 i, 2 i + 1 in the table for chunks of m tokens
template <bool kRev> __device__ __forceinline__ void fill_key_table(KeyTable& table, int i, int m, float l2, float add) {
  float w[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int tok = 2 * i + e;
    w[e] = tok < m ? add * exp2f((float)(kRev ? tok + 1 : m - 1 - tok) * l2) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    const uint32_t p = pack_bf16x2(w[0], w[1]);
    table.w[j][i] = p;
    w[0] -= bf16lo(p);
    w[1] -= bf16hi(p);
  }
}

// acc + a b for the low and the high halves of bf16 pairs a, b, in fp32: the mixed multiply-add takes bf16 operands
// as they lie, at full rate, where unpacking and conversion run at half
__device__ __forceinline__ float fma_lo(uint32_t a, uint32_t b, float acc) {
  float r;
  asm("{\n\t.reg .b16 al, ah, bl, bh;\n\tmov.b32 {al, ah}, %1;\n\tmov.b32 {bl, bh}, %2;\n\t"
      "fma.rn.f32.bf16 %0, al, bl, %3;\n\t}" : "=f"(r) : "r"(a), "r"(b), "f"(acc));
  return r;
}
__device__ __forceinline__ float fma_hi(uint32_t a, uint32_t b, float acc) {
  float r;
  asm("{\n\t.reg .b16 al, ah, bl, bh;\n\tmov.b32 {al, ah}, %1;\n\tmov.b32 {bl, bh}, %2;\n\t"
      "fma.rn.f32.bf16 %0, ah, bh, %3;\n\t}" : "=f"(r) : "r"(a), "r"(b), "f"(acc));
  return r;
}

// Two keys x times their factors w0 + w1 + w2 as kTerms bf16 terms.  x w0 = h + l exactly (both of 8 bits: h the
// rounded product, l what a multiply-add leaves of it); the second term is l + x w1 rounded once (2^-16 of the
// product is left, and x w2), the third what remains, formed in fp32.
template <int kTerms>
__device__ __forceinline__ void decay_pair(uint32_t xw, uint32_t w0, uint32_t w1, uint32_t w2, uint32_t (&term)[kTerms]) {
  auto b2 = [](uint32_t v) { return *reinterpret_cast<__nv_bfloat162*>(&v); };
  auto word = [](__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); };
  constexpr uint32_t kOne = 0x3f803f80u, kMinus = 0xbf80bf80u;
  const __nv_bfloat162 h = __hmul2_rn(b2(xw), b2(w0)), l = __hfma2(b2(xw), b2(w0), __hneg2(h));
  term[0] = word(h);
  term[1] = word(__hfma2(b2(xw), b2(w1), l));
  if constexpr (kTerms == 3) {
    const uint32_t lw = word(l);
    const float r0 = fma_lo(xw, w2, fma_lo(xw, w1, fma_lo(lw, kOne, fma_lo(term[1], kMinus, 0.f))));
    const float r1 = fma_hi(xw, w2, fma_hi(xw, w1, fma_hi(lw, kOne, fma_hi(term[1], kMinus, 0.f))));
    term[2] = pack_bf16x2(r0, r1);
  }
}

// The decayed keys of a chunk, transposed, as A operands (lane = channel, a column two tokens): 32 tokens from
// token 32 p of the 16 channels of a warp's quarter that `half` names.  Register 2 c + g of a thread holds tokens
// 32 p + 8 c + 2 (lane % 4) + {0, 1} of channel 8 g + lane / 4.  Tokens >= m become zero, whatever they hold.
template <int kTerms>
__device__ __forceinline__ void decayed_keys(const uint8_t* tile, const KeyTable& table, int p, int m, int quarter,
                                             int half, int lane, uint32_t (&key)[kTerms][8]) {
  uint32_t raw[8];
  const int c16 = 4 * quarter + 2 * half + ((lane >> 3) & 1);           // 16-byte chunk of the row
  const uint8_t* base = tile + (c16 >> 3) * 16384 + (((c16 & 7) ^ (lane & 7)) << 4) +
                        (32 * p + 8 * (lane >> 4) + (lane & 7)) * 128;
  tc::ldmatrix_x4_trans(base, raw);
  tc::ldmatrix_x4_trans(base + 2048, raw + 4);
  if (m < kC) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int tok = 32 * p + 8 * c + 2 * (lane & 3);
      const uint32_t keep = (tok < m ? 0xffffu : 0u) | (tok + 1 < m ? 0xffff0000u : 0u);
      raw[2 * c] &= keep;
      raw[2 * c + 1] &= keep;
    }
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int i = 16 * p + 4 * c + (lane & 3);
    const uint32_t w0 = table.w[0][i], w1 = table.w[1][i], w2 = kTerms == 3 ? table.w[2][i] : 0u;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      uint32_t term[kTerms];
      decay_pair<kTerms>(raw[2 * c + g], w0, w1, w2, term);
#pragma unroll
      for (int j = 0; j < kTerms; ++j) key[j][2 * c + g] = term[j];
    }
  }
}

// rows m .. 127 of a tile to zero: tokens behind the sequence, which may hold anything
__device__ __forceinline__ void zero_rows(uint8_t* tile, int m, int t, int nt) {
  for (int i = t; i < (kC - m) * 16; i += nt) {
    const int half = i >= (kC - m) * 8, r = i - half * (kC - m) * 8;
    *reinterpret_cast<uint4*>(tile + half * 16384 + m * 128 + r * 16) = make_uint4(0, 0, 0, 0);
  }
}

struct __align__(1024) ScanSmem {
  uint8_t y[2][kTile], z[2][kTile], x[2][kTile];   // two chunks
  uint8_t st[kTile];             // the state in bf16: rows y, columns z
  alignas(16) KeyTable key[2];   // factors of the decayed keys: full chunks, the early end's chunk
  alignas(16) float pd[64];      // lambda^{i - 32}, i >= 32
  uint64_t yz_full[2], x_full[2], x_free[2], o_full[2], staged[2], kd_ready[2], kd_free[2];
  uint64_t s_full, p_ready, far_done, o_free, u_full, s_ready, cleared, drain;
  uint32_t tmem_base;
  int abort, yz_issued, x_issued;
};
static_assert(sizeof(ScanSmem) + 1024 <= 232448, "shared memory of one CTA");

// TMEM columns.  The output accumulates the state's part first, which the near warps decay row by row.  P (bf16)
// overwrites part of X Y^T.  The decayed keys go by quarters of the chunk (32 tokens, 16 columns a term)
// through two slots, so that a quarter is made while another's product runs.
constexpr uint32_t kColP = 0, kColO = 128, kColKd = 256, kKdSlot = 64, kColU = 384;
// Block b of 32 tokens of P: blocks 0 and 1 over block 0 of X Y^T, 2 and 3 over block 2: what their warp has loaded
// before it stores them, so that no warp waits for another.
__device__ __forceinline__ constexpr uint32_t p_column(int b) { return kColP + 64 * (b >> 1) + 16 * (b & 1); }

// One row of a block of 32 columns of X Y^T times its weights, as bf16.  blocks: how many blocks it lies from the
// diagonal, base the decay to its nearest column.
template <bool kRev>
__device__ __forceinline__ void weigh_block(const uint32_t (&v)[32], uint32_t (&pk)[16], int blocks, float base,
                                            const float (&pd)[64], int lane) {
  if (blocks == 0) {
    // selected, not multiplied by zero: what is masked may be infinite
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float p[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int c = e + u;
        const float w = pd[kRev ? 32 + c - lane : 32 + lane - c];
        p[u] = (kRev ? c >= lane : c <= lane) ? __uint_as_float(v[c]) * w : 0.f;
      }
      pk[e / 2] = pack_bf16x2(p[0], p[1]);
    }
  } else {
    const float2 base2 = make_float2(base, base);
#pragma unroll
    for (int e = 0; e < 32; e += 4) {
      float4 w = *reinterpret_cast<const float4*>(&pd[kRev ? 32 + e : 60 - e]);
      if (!kRev) w = make_float4(w.w, w.z, w.y, w.x);
      const float2 p01 = __fmul2_rn(make_float2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                                    __fmul2_rn(base2, make_float2(w.x, w.y)));
      const float2 p23 = __fmul2_rn(make_float2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])),
                                    __fmul2_rn(base2, make_float2(w.z, w.w)));
      pk[e / 2] = pack_bf16x2(p01.x, p01.y);
      pk[e / 2 + 1] = pack_bf16x2(p23.x, p23.y);
    }
  }
}

// The first launch of a call clears the status word itself: a wait gives up after seconds, and the first block of
// the grid starts before any other has waited that long.
__device__ __forceinline__ void clear_status_word(uint32_t* status, int clear) {
  if (clear && blockIdx.x == 0 && threadIdx.x == 0) *status = 0;
}

// waits of the teardown go on after an abort (still bounded)
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  int zero = 0;
  tc::mbar_wait(bar, parity, &zero, nullptr);
}

}  // namespace

// One CTA per (batch, head, segment).  Warps 0-7 ("near"): P from X Y^T, then the output, two per token row;
// 8-23 ("state"): the decayed keys (each half of them two quarters of a chunk) and the state; then one for TMA
// loads, one for MMA issue and TMEM, one for TMA stores (waiting for a store to have read its tile would hold up P).
// The elementwise work is chains of dependent operations: many warps of few registers hide them.  The products run in the order X Y^T, X S^T, the keys' quarters, P Z, so that the keys' product and the
// state's update for the next chunk pass while P is made.
template <bool kRev, int kTerms>
__global__ void __launch_bounds__(kThreads, 1)
    k_decay_tc(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmY,
               const __grid_constant__ CUtensorMap tmZ, const __grid_constant__ CUtensorMap tmO, int B, int H, int T,
               int nseg, int seg_len, const float* __restrict__ decay, const int* __restrict__ lengths, const float* __restrict__ init,
               const float* __restrict__ seg_states, int transposed, float out_near, float out_ratio, float add,
               int clear, __nv_bfloat16* __restrict__ out, float* __restrict__ final, uint32_t* __restrict__ status,
               int clear_status) {
  clear_status_word(status, clear_status);
  const long long BH = (long long)B * H;
  const int seg = (int)(blockIdx.x / BH);
  const long long bh = blockIdx.x % BH;
  const int h = (int)(bh % H), b = (int)(bh / H);
  const int n_tok = decay_tokens(lengths, b, T);
  const int t0 = seg * seg_len, t1 = min(n_tok, t0 + seg_len);
  // the segment that ends the scan writes the final state, also where the sequence is empty
  const int last_seg = kRev || n_tok == 0 ? 0 : (n_tok - 1) / seg_len;
  const bool write_final = final != nullptr && seg == last_seg;
  const int nch = t1 > t0 ? (t1 - t0 + kC - 1) / kC : 0;
  // rows of the segment behind the sequence to zero, if asked for
  auto clear_behind = [&] {
    const int c0 = max(t0, t1), c1 = min(T, t0 + seg_len);
    if (clear)
      for (int i = threadIdx.x; i < (c1 - c0) * 16; i += kThreads)
        *reinterpret_cast<uint4*>(out + (((long long)b * T + c0 + (i >> 4)) * H + h) * 128 + 8 * (i & 15)) =
            make_uint4(0, 0, 0, 0);
  };
  if (nch == 0 && !write_final) {
    clear_behind();
    return;
  }
  const float* src = nseg > 1 ? seg_states + ((long long)seg * BH + bh) * 16384 : init ? init + bh * 16384 : nullptr;

  extern __shared__ uint8_t smem_raw[];
  ScanSmem& sm = tc::smem_align<ScanSmem>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &sm.abort;
  const float lambda = decay[h], l2 = decay_log2(lambda);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.yz_full[i], 1);
      tc::mbar_init(&sm.x_full[i], 1);
      tc::mbar_init(&sm.x_free[i], 1);
      tc::mbar_init(&sm.o_full[i], 1);
      tc::mbar_init(&sm.staged[i], kNearWarps);
      tc::mbar_init(&sm.kd_ready[i], kStateWarps / 2);
      tc::mbar_init(&sm.kd_free[i], 1);
    }
    tc::mbar_init(&sm.s_full, 1);
    tc::mbar_init(&sm.p_ready, kNearWarps);
    tc::mbar_init(&sm.far_done, 1);
    tc::mbar_init(&sm.o_free, kNearWarps);
    tc::mbar_init(&sm.u_full, 1);
    tc::mbar_init(&sm.s_ready, kStateWarps);
    tc::mbar_init(&sm.cleared, kNearWarps);
    tc::mbar_init(&sm.drain, 1);
    sm.abort = 0;
    sm.yz_issued = sm.x_issued = 0;
    tc::fence_barrier_init();
  }
  if (tid >= 64 && tid < 128) sm.pd[tid - 64] = tid < 96 ? 0.f : exp2f((float)(tid - 96) * l2);
  if (tid >= 128 && tid < 256) {
    const int early = (tid >> 6) & 1;
    fill_key_table<kRev>(sm.key[early], tid & 63, early ? (t1 - t0) % kC : kC, l2, add);
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&sm.tmem_base, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  // chunk n of the scan order: its first token and its valid rows
  auto chunk_t = [&](int n) { return t0 + kC * (kRev ? nch - 1 - n : n); };
  auto chunk_m = [&](int n) { return min(kC, t1 - chunk_t(n)); };
  // whether the state is read for chunk n, and whether its update is made (by all chunks but the last, if at all)
  auto has_state = [&](int n) { return n > 0 || src != nullptr; };
  auto carries = [&](int n) { return n + 1 < nch || write_final; };

  // whole chunks leave by TMA, and so does one that ends at T, where the tensor map cuts it off; rows behind a shorter
  // sequence stay as they were
  auto by_tma = [&](int n) { return chunk_m(n) == kC || chunk_t(n) + chunk_m(n) == T; };

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------ TMA
    // chunk n over chunk n - 2: Y and Z once its last product is done, X once its output has left
    if (lane == 0) {
      auto load = [&](const CUtensorMap* tm, uint64_t* bar, uint8_t* dst, int n) {
        tc::tma_load_4d(tm, bar, dst, 0, h, chunk_t(n), b);
        tc::tma_load_4d(tm, bar, dst + 16384, 64, h, chunk_t(n), b);
      };
      for (int n = 0; n < nch; ++n) {
        const int i = n & 1, before = ((n >> 1) - 1) & 1;
        if (n > 1 && !tc::mbar_wait(&sm.o_full[i], before, abort_flag, status)) break;
        tc::mbar_arrive_expect_tx(&sm.yz_full[i], 2 * kTile);
        load(&tmY, &sm.yz_full[i], sm.y[i], n);
        load(&tmZ, &sm.yz_full[i], sm.z[i], n);
        sm.yz_issued = n + 1;
        if (n > 1 && !tc::mbar_wait(&sm.x_free[i], before, abort_flag, status)) break;
        tc::mbar_arrive_expect_tx(&sm.x_full[i], kTile);
        load(&tmX, &sm.x_full[i], sm.x[i], n);
        sm.x_issued = n + 1;
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ MMA
    if (lane == 0) {
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) { return ok = ok && tc::mbar_wait(bar, parity, abort_flag, status); };
      const uint32_t as = tc::smem_u32(sm.st);
      for (int n = 0; n < nch && ok; ++n) {
        const int i = n & 1, pair = (n >> 1) & 1;
        const uint32_t ay = tc::smem_u32(sm.y[i]), ax = tc::smem_u32(sm.x[i]), az = tc::smem_u32(sm.z[i]);
        if (!wait(&sm.yz_full[i], pair) || !wait(&sm.x_full[i], pair)) break;
        if (kRev && n == 0 && chunk_m(0) < kC && !wait(&sm.cleared, 0)) break;
        tc::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          tc::umma_bf16(tmem + kColP, tc::smem_desc(ax + off, 16, 1024), tc::smem_desc(ay + off, 16, 1024), kIdescKK,
                        kk > 0 ? 1u : 0u);
        }
        tc::umma_commit(&sm.s_full);
        if (!wait(&sm.s_ready, n & 1)) break;
        if (n > 0 && !wait(&sm.o_free, (n - 1) & 1)) break;
        tc::tc_fence_after();
        if (has_state(n)) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            tc::umma_bf16(tmem + kColO, tc::smem_desc(ax + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024),
                          tc::smem_desc(as + kk * 2048, 16384, 1024), kIdescKM, kk > 0 ? 1u : 0u);
        }
        tc::umma_commit(&sm.far_done);
        // where the chunk ends early, Z's rows behind it are cleared before p_ready
        if (!kRev && chunk_m(n) < kC && !wait(&sm.p_ready, n & 1)) break;
        if (carries(n)) {
#pragma unroll
          for (int quarter = 0; quarter < 4; ++quarter) {
            const int slot = quarter & 1;
            if (!wait(&sm.kd_ready[slot], quarter >> 1)) break;      // two uses of a slot per chunk
            tc::tc_fence_after();
#pragma unroll
            for (int term = 0; term < kTerms; ++term)
#pragma unroll
              for (int kk = 0; kk < 2; ++kk)
                tc::umma_bf16_ts(tmem + kColU, tmem + kColKd + kKdSlot * slot + 16 * term + 8 * kk,
                                 tc::smem_desc(az + (2 * quarter + kk) * 2048, 16384, 1024), kIdescKM,
                                 quarter + term + kk > 0 ? 1u : 0u);
            tc::umma_commit(&sm.kd_free[slot]);
          }
          if (!ok) break;
          tc::umma_commit(&sm.u_full);
        }
        if (!wait(&sm.p_ready, n & 1)) break;
        tc::tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc::umma_bf16_ts(tmem + kColO, tmem + p_column(kk >> 1) + 8 * (kk & 1), tc::smem_desc(az + kk * 2048, 16384, 1024), kIdescKM,
                           has_state(n) || kk > 0 ? 1u : 0u);
        tc::umma_commit(&sm.o_full[i]);
      }
    }
  } else if (warp == kStoreWarp) {
    // ------------------------------------------------------------ stores of the staged output
    if (lane == 0) {
      for (int n = 0; n < nch; ++n) {
        const int i = n & 1, t = chunk_t(n);
        if (!tc::mbar_wait(&sm.staged[i], (n >> 1) & 1, abort_flag, status)) break;
        if (by_tma(n)) {
          tc::tma_store_4d(&tmO, sm.x[i], 0, h, t, b);
          tc::tma_store_4d(&tmO, sm.x[i] + 16384, 64, h, t, b);
          tc::bulk_commit();
          tc::bulk_wait_read_all();
        }
        tc::mbar_arrive(&sm.x_free[i]);
      }
      tc::bulk_wait_all();
    }
  } else if (warp < kNearWarps) {
    // ------------------------------------------------------------ near terms and output
    const int quarter = warp & 3, half = warp >> 2;     // this warp's 64 columns: half
    const int r = 32 * quarter + lane;                  // token of the chunk = TMEM lane
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    // lambda^{distance} off the diagonal blocks = lambda^{distance of the block's nearest column} times
    // lambda^{the columns between}
    const float nearest = exp2f((float)(kRev ? 32 - lane : lane + 1) * l2), pass = exp2f(32.f * l2);
    bool ok = true;
    // In reverse the tokens behind the sequence are not masked by their place: Y and Z rows of the first chunk are
    // cleared before its first product (the warps that decay the keys mask theirs, cleared or not).  Masking the
    // weights instead put a second form of them into the loop, which cost every chunk (73 against 68 us for 12288
    // tokens x 24 heads).
    if (kRev && nch > 0 && chunk_m(0) < kC && (ok = tc::mbar_wait(&sm.yz_full[0], 0, abort_flag, status))) {
      zero_rows(sm.y[0], chunk_m(0), tid, 32 * kNearWarps);
      zero_rows(sm.z[0], chunk_m(0), tid, 32 * kNearWarps);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.cleared);
    }
    for (int n = 0; n < nch && ok; ++n) {
      const int m = chunk_m(n), i = n & 1, pair = (n >> 1) & 1;
      if (!(ok = tc::mbar_wait(&sm.s_full, n & 1, abort_flag, status))) break;
      tc::tc_fence_after();
#pragma unroll 1
      for (int q = 0; q < 2; ++q) {
        const int cb = 2 * half + q;                    // block of 32 columns
        const int blocks = kRev ? cb - quarter : quarter - cb;           // 0 (diagonal) .. 3
        uint32_t pk[16];
        if (blocks < 0) {                               // no token of the block is in reach
#pragma unroll
          for (int e = 0; e < 16; ++e) pk[e] = 0;
        } else {
          uint32_t v[32];
          tc::tmem_ld32(tmem + kColP + 32 * cb + lane_off, v);
          tc::tmem_ld_wait();
          const float base = blocks == 1 ? nearest : blocks == 2 ? nearest * pass : nearest * pass * pass;
          weigh_block<kRev>(v, pk, blocks, base, sm.pd, lane);
        }
        tc::tmem_st16(tmem + p_column(cb) + lane_off, pk);
      }
      if (has_state(n)) {     // the state's part of the output, in units of out_near
        if (!(ok = tc::mbar_wait(&sm.far_done, n & 1, abort_flag, status))) break;
        tc::tc_fence_after();
        const float wf = out_ratio * exp2f((float)(kRev ? m - 1 - r : r + 1) * l2);
        const float2 wf2 = make_float2(wf, wf);
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          const uint32_t at = tmem + kColO + 32 * (2 * half + part) + lane_off;
          uint32_t f[32];
          tc::tmem_ld32(at, f);
          tc::tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 y = __fmul2_rn(make_float2(__uint_as_float(f[e]), __uint_as_float(f[e + 1])), wf2);
            f[e] = __float_as_uint(y.x);
            f[e + 1] = __float_as_uint(y.y);
          }
          tc::tmem_st32(at, f);
        }
      }
      tc::tmem_st_wait();
      if (!kRev && m < kC) {              // the last chunk; in reverse, where it is the first, all is done before
        if (!(ok = tc::mbar_wait(&sm.yz_full[i], pair, abort_flag, status))) break;
        zero_rows(sm.z[i], m, tid, 32 * kNearWarps);
        tc::fence_proxy_async_smem();
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.p_ready);
      if (!(ok = tc::mbar_wait(&sm.o_full[i], pair, abort_flag, status))) break;
      tc::tc_fence_after();
      // the X tile has been read (its products come before the one that o_full follows): it stages the output
      uint8_t* stage = sm.x[i];
#pragma unroll 1
      for (int part = 0; part < 2; ++part) {
        uint32_t a[32];
        tc::tmem_ld32(tmem + kColO + 32 * (2 * half + part) + lane_off, a);
        tc::tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          uint32_t w[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float2 y = __fmul2_rn(make_float2(__uint_as_float(a[e + 2 * u]), __uint_as_float(a[e + 2 * u + 1])),
                                        make_float2(out_near, out_near));
            w[u] = pack_bf16x2(y.x, y.y);
          }
          *reinterpret_cast<uint4*>(stage + tile_chunk(r, 4 * (2 * half + part) + e / 8)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.o_free);
      if (by_tma(n)) {
        tc::fence_proxy_async_smem();
      } else {
        // this warp's own rows and columns, eight lanes per row: a barrier with the other warps could wait for one that
        // has left its role after a wait ran out
        const int t = chunk_t(n), c = 8 * half + (lane & 7);
#pragma unroll 4
        for (int row = 32 * quarter + (lane >> 3); row < min(m, 32 * quarter + 32); row += 4)
          *reinterpret_cast<uint4*>(out + (((long long)b * T + t + row) * H + h) * 128 + 8 * c) =
              *reinterpret_cast<const uint4*>(stage + tile_chunk(row, c));
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.staged[i]);
    }
  } else {
    // ------------------------------------------------------------ state
    const int quarter = warp & 3, sub = (warp - kNearWarps) >> 2;
    const int k = 32 * quarter + lane;                  // y channel = TMEM lane
    const int v0 = 32 * sub;                            // z channels v0 .. v0 + 31
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    float2 s[16];                                       // S[v0 + 2 p][k], S[v0 + 2 p + 1][k]
    if (!src) {
#pragma unroll
      for (int p = 0; p < 16; ++p) s[p] = make_float2(0.f, 0.f);
    } else if (transposed) {
#pragma unroll
      for (int p = 0; p < 16; p += 2) {
        const float4 f = *reinterpret_cast<const float4*>(src + k * 128 + v0 + 2 * p);
        s[p] = make_float2(f.x, f.y);
        s[p + 1] = make_float2(f.z, f.w);
      }
    } else {
#pragma unroll
      for (int p = 0; p < 16; ++p)
        s[p] = make_float2(src[(v0 + 2 * p) * 128 + k], src[(v0 + 2 * p + 1) * 128 + k]);
    }
    auto publish = [&]() {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4*>(sm.st + tile_chunk(k, 4 * sub + c)) =
            make_uint4(pack_bf16x2(s[4 * c].x, s[4 * c].y), pack_bf16x2(s[4 * c + 1].x, s[4 * c + 1].y),
                       pack_bf16x2(s[4 * c + 2].x, s[4 * c + 2].y), pack_bf16x2(s[4 * c + 3].x, s[4 * c + 3].y));
      tc::fence_proxy_async_smem();
    };
    // this warp's part of quarter 2 use + slot of chunk n's keys: 16 channels, 32 tokens
    const int slot = sub >> 1, half = sub & 1;
    auto keys = [&](int n, int use) -> bool {
      const int m = chunk_m(n), i = n & 1;
      if (!tc::mbar_wait(&sm.yz_full[i], (n >> 1) & 1, abort_flag, status)) return false;
      uint32_t key[kTerms][8];
      decayed_keys(sm.y[i], sm.key[m < kC], 2 * use + slot, m, quarter, half, lane, key);
      // the slot's use before this one has been read
      if (n + use > 0 && !tc::mbar_wait(&sm.kd_free[slot], use ^ 1, abort_flag, status)) return false;
      tc::tc_fence_after();
      const uint32_t at = tmem + lane_off + ((uint32_t)(16 * half) << 16) + kColKd + kKdSlot * slot;
#pragma unroll
      for (int j = 0; j < kTerms; ++j) tc::tmem_st16x128b_x4(at + 16 * j, key[j]);
      tc::tmem_st_wait();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.kd_ready[slot]);
      return true;
    };
    bool ok = true;
    if (nch > 0) {
      if (src) publish();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.s_ready);
    }
    // keys (0, 0), (0, 1), (1, 0), update 0, (1, 1), (2, 0), update 1, ..: a chunk's first keys are made while the
    // product of the chunk before runs.  One instance of each in the code: it is fetched more slowly than it runs.
    for (int i = 0; ok; ++i) {
      const int n = i >> 1, use = i & 1;
      const bool more = n < nch && carries(n);
      if (more && !(ok = keys(n, use))) break;
      if (use == 0 && n > 0) {
        const float keep = exp2f((float)chunk_m(n - 1) * l2);
        if (!(ok = tc::mbar_wait(&sm.u_full, (n - 1) & 1, abort_flag, status))) break;
        tc::tc_fence_after();
        uint32_t u[32];
        tc::tmem_ld32(tmem + kColU + v0 + lane_off, u);
        tc::tmem_ld_wait();
#pragma unroll
        for (int p = 0; p < 16; ++p)
          s[p] = __ffma2_rn(s[p], make_float2(keep, keep), make_float2(__uint_as_float(u[2 * p]), __uint_as_float(u[2 * p + 1])));
        if (n < nch) {
          if (!(ok = tc::mbar_wait(&sm.far_done, (n - 1) & 1, abort_flag, status))) break;   // the old state has been read
          publish();
          tc::tc_fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&sm.s_ready);
        }
      }
      if (!more) break;
    }
    if (write_final && ok) {
      float* dst = final + bh * 16384;
      if (transposed) {
#pragma unroll
        for (int p = 0; p < 16; p += 2)
          *reinterpret_cast<float4*>(dst + k * 128 + v0 + 2 * p) = make_float4(s[p].x, s[p].y, s[p + 1].x, s[p + 1].y);
      } else {
#pragma unroll
        for (int p = 0; p < 16; ++p) {
          dst[(v0 + 2 * p) * 128 + k] = s[p].x;
          dst[(v0 + 2 * p + 1) * 128 + k] = s[p].y;
        }
      }
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (sm.abort && warp == kMmaWarp && lane == 0) {   // no product may run on, whichever warp gave up
    tc::umma_commit(&sm.drain);
    drain_wait(&sm.drain, 0);
  }
  if (sm.abort && tid == 0) {   // no copy may land after the CTA has left
    for (int n = max(0, sm.yz_issued - 2); n < sm.yz_issued; ++n) drain_wait(&sm.yz_full[n & 1], (n >> 1) & 1);
    for (int n = max(0, sm.x_issued - 2); n < sm.x_issued; ++n) drain_wait(&sm.x_full[n & 1], (n >> 1) & 1);
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
  clear_behind();
}

// ---------------------------------------------------------------- states of the segments
// The state that a segment's own tokens leave at its end: the scan's state part alone.  Bound by the warps' work on the
// keys with three terms (2950 cycles per chunk, products 51 % of them), by them and DRAM (58 % of its rate) with two:
// 30 us and 26 - 29 us for 12288 tokens x 24 heads.  Bringing later chunks into L2 ahead of their loads is slower, here and
// in the scan (two chunks ahead: 32 and 60 us; four: 35 and 77), and so is one instance of `keys` for both halves (33).
namespace {

constexpr int kSegStages = 3;
constexpr int kSegWarps = 16;
constexpr int kSegThreads = 32 * (kSegWarps + 2);
struct __align__(1024) SegSmem {
  uint8_t y[kSegStages][kTile], z[kSegStages][kTile];
  alignas(16) KeyTable key[2];
  uint64_t full[kSegStages], empty[kSegStages], kd_ready[2], kd_free[2], u_full[2], u_free[2], drain;
  uint32_t tmem_base;
  int abort, issued;
};
// TMEM columns: two sets of the keys' product (chunks alternate), then the keys of the two halves of a chunk
constexpr uint32_t kSegColKd = 256, kSegKdCols = 128;

}  // namespace

template <bool kRev, int kTerms>
__global__ void __launch_bounds__(kSegThreads, 1)
    k_decay_segments_tc(const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmZ, int B, int H,
                        int T, int seg_len, const float* __restrict__ decay, const int* __restrict__ lengths,
                        float add, float* __restrict__ states, uint32_t* __restrict__ status, int clear_status) {
  clear_status_word(status, clear_status);
  const long long BH = (long long)B * H;
  const int seg = (int)(blockIdx.x / BH) + (kRev ? 1 : 0);   // nothing follows the order's last segment
  const long long bh = blockIdx.x % BH;
  const int h = (int)(bh % H), b = (int)(bh / H);
  const int t0 = seg * seg_len, t1 = min(decay_tokens(lengths, b, T), t0 + seg_len);
  if (t1 <= t0) return;                       // the prefix reads no state of an empty segment
  const int nch = (t1 - t0 + kC - 1) / kC;
  extern __shared__ uint8_t smem_raw[];
  SegSmem& sm = tc::smem_align<SegSmem>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  volatile int* abort_flag = &sm.abort;
  const float l2 = decay_log2(decay[h]);
  if (tid == 0) {
    for (int s = 0; s < kSegStages; ++s) {
      tc::mbar_init(&sm.full[s], 1);
      tc::mbar_init(&sm.empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      tc::mbar_init(&sm.kd_ready[s], kSegWarps);
      tc::mbar_init(&sm.kd_free[s], 1);
      tc::mbar_init(&sm.u_full[s], 1);
      tc::mbar_init(&sm.u_free[s], kSegWarps);
    }
    tc::mbar_init(&sm.drain, 1);
    sm.abort = 0;
    sm.issued = 0;
    tc::fence_barrier_init();
  }
  if (tid < 128) fill_key_table<kRev>(sm.key[tid >> 6], tid & 63, tid >> 6 ? (t1 - t0) % kC : kC, l2, add);
  if (warp == kSegWarps + 1) {
    tc::tmem_alloc(&sm.tmem_base, 512);
    tc::tmem_relinquish();
  }
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tmem = sm.tmem_base;

  if (warp == kSegWarps) {
    if (lane == 0) {
      for (int n = 0; n < nch; ++n) {
        const int s = n % kSegStages, t = t0 + kC * (kRev ? nch - 1 - n : n);
        if (!tc::mbar_wait(&sm.empty[s], ((n / kSegStages) & 1) ^ 1, abort_flag, status)) break;
        tc::mbar_arrive_expect_tx(&sm.full[s], 2 * kTile);
        tc::tma_load_4d(&tmY, &sm.full[s], sm.y[s], 0, h, t, b);
        tc::tma_load_4d(&tmY, &sm.full[s], sm.y[s] + 16384, 64, h, t, b);
        tc::tma_load_4d(&tmZ, &sm.full[s], sm.z[s], 0, h, t, b);
        tc::tma_load_4d(&tmZ, &sm.full[s], sm.z[s] + 16384, 64, h, t, b);
        sm.issued = n + 1;
      }
    }
  } else if (warp == kSegWarps + 1) {
    if (lane == 0) {
      bool ok = true;
      for (int n = 0; n < nch; ++n) {
        const int s = n % kSegStages, ub = n & 1;
        const uint32_t az = tc::smem_u32(sm.z[s]);
        if (n > 1 && !(ok = tc::mbar_wait(&sm.u_free[ub], ((n >> 1) - 1) & 1, abort_flag, status))) break;
#pragma unroll
        for (int part = 0; part < 2 && ok; ++part) {
          if (!(ok = tc::mbar_wait(&sm.kd_ready[part], n & 1, abort_flag, status))) break;
          tc::tc_fence_after();
#pragma unroll
          for (int i = 0; i < 4 * kTerms; ++i)
            tc::umma_bf16_ts(tmem + 128 * ub, tmem + kSegColKd + kSegKdCols * part + 8 * i,
                             tc::smem_desc(az + (4 * part + (i & 3)) * 2048, 16384, 1024), kIdescKM,
                             part + i > 0 ? 1u : 0u);
          tc::umma_commit(&sm.kd_free[part]);
        }
        if (!ok) break;
        tc::umma_commit(&sm.u_full[ub]);
        tc::umma_commit(&sm.empty[s]);
      }
    }
  } else {
    // half by half, the keys are made while the product of the half before runs; a warp takes 16 channels, 32 tokens
    const int quarter = warp & 3, sub = warp >> 2, v0 = 32 * sub;
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    auto chunk_t = [&](int n) { return t0 + kC * (kRev ? nch - 1 - n : n); };
    auto keys = [&](int n, int part) -> bool {
      const int s = n % kSegStages, m = min(kC, t1 - chunk_t(n));
      uint32_t key[kTerms][8];
      decayed_keys(sm.y[s], sm.key[m < kC], 2 * part + (sub >> 1), m, quarter, sub & 1, lane, key);
      if (n > 0 && !tc::mbar_wait(&sm.kd_free[part], (n - 1) & 1, abort_flag, status)) return false;
      tc::tc_fence_after();
      const uint32_t kd = tmem + kSegColKd + kSegKdCols * part + lane_off + ((uint32_t)(16 * (sub & 1)) << 16) + 16 * (sub >> 1);
#pragma unroll
      for (int i = 0; i < kTerms; ++i) tc::tmem_st16x128b_x4(kd + 32 * i, key[i]);
      tc::tmem_st_wait();
      if (part == 0 && m < kC) {
        zero_rows(sm.z[s], m, tid, 32 * kSegWarps);
        tc::fence_proxy_async_smem();
      }
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.kd_ready[part]);
      return true;
    };
    float2 acc[16];                                     // [v0 + 2 p], [v0 + 2 p + 1] of y channel 32 quarter + lane
#pragma unroll
    for (int p = 0; p < 16; ++p) acc[p] = make_float2(0.f, 0.f);
    auto take = [&](int n) -> bool {                    // acc <- lambda^{tokens} acc + the product of chunk n
      const int ub = n & 1;
      const float keep = exp2f((float)min(kC, t1 - chunk_t(n)) * l2);
      if (!tc::mbar_wait(&sm.u_full[ub], (n >> 1) & 1, abort_flag, status)) return false;
      tc::tc_fence_after();
      uint32_t u[32];
      tc::tmem_ld32(tmem + 128 * ub + v0 + lane_off, u);
      tc::tmem_ld_wait();
#pragma unroll
      for (int p = 0; p < 16; ++p)
        acc[p] = __ffma2_rn(acc[p], make_float2(keep, keep), make_float2(__uint_as_float(u[2 * p]), __uint_as_float(u[2 * p + 1])));
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sm.u_free[ub]);
      return true;
    };
    bool ok = true;
    for (int n = 0; n < nch && ok; ++n) {
      ok = tc::mbar_wait(&sm.full[n % kSegStages], (n / kSegStages) & 1, abort_flag, status) && keys(n, 0) && keys(n, 1) &&
           (n == 0 || take(n - 1));
    }
    if (ok && take(nch - 1)) {
      float* dst = states + ((long long)seg * BH + bh) * 16384 + v0 * 128 + 32 * quarter + lane;   // [z][y]
#pragma unroll
      for (int p = 0; p < 16; ++p) {
        dst[2 * p * 128] = acc[p].x;
        dst[(2 * p + 1) * 128] = acc[p].y;
      }
    }
  }

  tc::tc_fence_before();
  __syncthreads();
  if (sm.abort && warp == kSegWarps + 1 && lane == 0) {
    tc::umma_commit(&sm.drain);
    drain_wait(&sm.drain, 0);
  }
  if (sm.abort && tid == 0) {
    const int issued = sm.issued;
    for (int s = 0; s < kSegStages && s < issued; ++s) {
      const int n = s + (issued - 1 - s) / kSegStages * kSegStages;
      drain_wait(&sm.full[s], (n / kSegStages) & 1);
    }
  }
  __syncthreads();
  if (warp == kSegWarps + 1) {
    tc::tc_fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

namespace {
// once per kernel and device
template <typename K> cudaError_t smem_opt_in(K kernel, size_t bytes, std::atomic<unsigned long long>& done) {
  int dev;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && (done.load() >> dev & 1))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ULL << dev);
  return e;
}
}  // namespace

cudaError_t launch_decay_scan_tc(const DecayScan& s, const DecayPlan& p) {
  CUtensorMap tx, ty, tz, to;
  if (!tmap_tokens_bf16(&tx, s.x, 128, s.H, s.T, s.B, kC) || !tmap_tokens_bf16(&ty, s.y, 128, s.H, s.T, s.B, kC) ||
      !tmap_tokens_bf16(&tz, s.z, 128, s.H, s.T, s.B, kC) || !tmap_tokens_bf16(&to, s.out, 128, s.H, s.T, s.B, kC))
    return cudaErrorInvalidValue;
  const size_t smem = sizeof(ScanSmem) + 1024;
  auto kern = s.exact_state ? (s.reverse ? k_decay_tc<true, 3> : k_decay_tc<false, 3>)
                            : (s.reverse ? k_decay_tc<true, 2> : k_decay_tc<false, 2>);
  static std::atomic<unsigned long long> done[4];
  cudaError_t e = smem_opt_in(kern, smem, done[2 * s.exact_state + s.reverse]);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)((long long)s.B * s.H * p.nseg), kThreads, smem, s.stream>>>(
      tx, ty, tz, to, s.B, s.H, s.T, p.nseg, p.len, s.decay, s.lengths, s.init, s.seg_states, s.transposed ? 1 : 0,
      s.out_near, s.out_far / s.out_near, s.add, s.clear ? 1 : 0, static_cast<__nv_bfloat16*>(s.out), s.final, s.status,
      s.clear_status ? 1 : 0);
  return cudaGetLastError();
}

cudaError_t launch_decay_segments_tc(const DecayScan& s, const DecayPlan& p, float* states) {
  CUtensorMap ty, tz;
  if (!tmap_tokens_bf16(&ty, s.y, 128, s.H, s.T, s.B, kC) || !tmap_tokens_bf16(&tz, s.z, 128, s.H, s.T, s.B, kC))
    return cudaErrorInvalidValue;
  const size_t smem = sizeof(SegSmem) + 1024;
  auto kern = s.exact_state ? (s.reverse ? k_decay_segments_tc<true, 3> : k_decay_segments_tc<false, 3>)
                            : (s.reverse ? k_decay_segments_tc<true, 2> : k_decay_segments_tc<false, 2>);
  static std::atomic<unsigned long long> done[4];
  cudaError_t e = smem_opt_in(kern, smem, done[2 * s.exact_state + s.reverse]);
  if (e != cudaSuccess) return e;
  kern<<<(unsigned)((long long)s.B * s.H * (p.nseg - 1)), kSegThreads, smem, s.stream>>>(
      ty, tz, s.B, s.H, s.T, p.len, s.decay, s.lengths, s.add, states, s.status, s.clear_status ? 1 : 0);
  return cudaGetLastError();
}

}  // namespace vdn
