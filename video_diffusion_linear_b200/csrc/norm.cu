// Layer norm, forward and backward, over the last axis of [rows, groups, d], weight and bias [groups, d]
// (groups = 1: shared by every row; groups = heads: the norm of a read-out).
//
//   mu = mean x, rstd = (mean (x - mu)^2 + eps)^-1/2, xh = (x - mu) rstd, y = xh w + b
//   g = dy w:  dx = rstd (g - mean g - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Bound by the bytes of x, y (dy, dx): each is read or written once.  A team of threads holds a whole row
// (in registers, but for the spills named below), so the variance is taken about the mean in a second sweep (no
// sum-of-squares cancellation).  A block walks rows of one group, so that a thread meets the same columns in
// all of them: weight and bias stay in registers, and in the backward its part of dw and db too; blocks leave
// partial sums that a second kernel adds in a fixed order.  A row's vectors are requested while the row before is
// worked on, and lines of the rows after that are brought into L2 (48360 x 24 rows of 128, bf16: 13 % off the forward
// and the backward).  Small teams with two (fp32: four) vectors per thread beat a team twice as large with one:
// fewer shuffles, and fewer addresses per element, which is what the kernels issue besides the arithmetic.
//
// All accesses are 16-byte vectors, whatever the width: where a row does not start on 16 bytes, the
// vectors start before it (`shift` elements, cleared), and a block takes rows of one shift only -- every kVec-th
// -- so that its columns stay in place.  Vectors that reach outside a row are stored by elements, and one
// that would reach past the tensor's end is loaded by elements.
//
// Measured with a cold L2 and buffers given, 48360 x 24 rows of 128: bf16 forward 102 us, 5.8 TB/s, backward 169 us,
// 5.3 TB/s; fp32 190 us, 6.2 TB/s, and 310 us, 5.7 TB/s.
//
// Spilled bytes a thread (stores): forward none up to 8192 wide, beyond (teams of 1024, 64 registers) 84 - 516; backward
// bf16 none at the widths of whole teams and 8 - 80 at others, fp32 12 - 124 and 68 - 276, beyond 8192 up to 1128.  They
// cost the long rows most: 3000 rows of 16384, fp32, take 162 us and 366 us (2.4 and 1.6 TB/s); 3000 of 8192, bf16,
// 33 us and 52 us (3.0 and 2.8 TB/s).
#include <cmath>

#include "check.h"
#include "common.cuh"
#include "internal.h"

namespace vdn {
namespace {

constexpr int kNormMaxWidth = 16384;
constexpr int kAhead = 3;               // rows ahead of the one worked on that are brought into L2
constexpr int kBlock = 256;             // threads of a block, unless a team is larger

template <typename T> constexpr int kVecOf = 16 / (int)sizeof(T);

// the 16 bytes of a vector as pairs of floats
template <typename T> __device__ __forceinline__ void unpack(const uint4& a, float2 (&v)[kVecOf<T> / 2]) {
  if constexpr (sizeof(T) == 4) {
    v[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
    v[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
  } else {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = make_float2(bf16lo(w[e]), bf16hi(w[e]));
  }
}
template <typename T> __device__ __forceinline__ uint4 pack(const float2 (&v)[kVecOf<T> / 2]) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(v[0].x), __float_as_uint(v[0].y), __float_as_uint(v[1].x), __float_as_uint(v[1].y));
  else
    return make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y),
                      pack_bf16x2(v[3].x, v[3].y));
}
// a line that a later row will want, into L2: more in flight than registers could hold
__device__ __forceinline__ void prefetch_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Columns c .. c + kVec - 1 of the row at `row` (element index of its column 0); c + row is a multiple of kVec.
// Elements outside the row hold whatever lies there (load) or are left alone (store).
template <typename T> __device__ __forceinline__ uint4 load_cols(const T* p, long long row, int c, int d, long long total) {
  if (row + c + kVecOf<T> <= total) return *reinterpret_cast<const uint4*>(p + row + c);
  uint32_t w[4] = {0, 0, 0, 0};              // the tensor's last elements
  for (int e = c < 0 ? -c : 0; c + e < d; ++e) {
    if constexpr (sizeof(T) == 4) w[e] = __float_as_uint(p[row + c + e]);
    else w[e / 2] |= (uint32_t)__bfloat16_as_ushort(p[row + c + e]) << (16 * (e & 1));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// zero in their place, where the vector is used (not where it is requested, which would wait for it)
template <typename T> __device__ __forceinline__ uint4 clear_outside(uint4 a, int c, int d) {
  if (c >= 0 && c + kVecOf<T> <= d) return a;
  uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int e = 0; e < kVecOf<T>; ++e) {
    const uint32_t bits = sizeof(T) == 4 ? 0xffffffffu : e & 1 ? 0xffff0000u : 0xffffu;
    if (c + e < 0 || c + e >= d) w[e * (int)sizeof(T) / 4] &= ~bits;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T> __device__ __forceinline__ void store_cols(T* p, long long row, int c, int d, const float2 (&v)[kVecOf<T> / 2]) {
  if (c >= 0 && c + kVecOf<T> <= d) {
    *reinterpret_cast<uint4*>(p + row + c) = pack<T>(v);
  } else {
#pragma unroll
    for (int e = 0; e < kVecOf<T>; ++e)
      if (c + e >= 0 && c + e < d) p[row + c + e] = from_f32<T>(e & 1 ? v[e / 2].y : v[e / 2].x);
  }
}
// the parameters of columns c .. c + kVec - 1 (`p`: the group's row of them, NULL: `otherwise`)
template <int kVec> __device__ __forceinline__ void load_par(const float* p, int c, int d, float otherwise, float2 (&v)[kVec / 2]) {
#pragma unroll
  for (int e = 0; e < kVec / 2; ++e) v[e] = make_float2(otherwise, otherwise);
  if (!p) return;
  if (c >= 0 && c + kVec <= d && (uintptr_t)(p + c) % 16 == 0) {
#pragma unroll
    for (int e = 0; e < kVec / 2; e += 2) {
      const float4 f = *reinterpret_cast<const float4*>(p + c + 2 * e);
      v[e] = make_float2(f.x, f.y);
      v[e + 1] = make_float2(f.z, f.w);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kVec / 2; ++e) {
      if (c + 2 * e >= 0 && c + 2 * e < d) v[e].x = p[c + 2 * e];
      if (c + 2 * e + 1 >= 0 && c + 2 * e + 1 < d) v[e].y = p[c + 2 * e + 1];
    }
  }
}
// v where columns c, c + 1 lie in the row, zero elsewhere (selected: a neighbour's element may be anything)
__device__ __forceinline__ float2 inside(float2 v, int c, int d) {
  return make_float2(c >= 0 && c < d ? v.x : 0.f, c + 1 >= 0 && c + 1 < d ? v.y : 0.f);
}

// sums over the kTeam threads of a row; every thread gets them.  Teams above a warp meet in `red` (two
// alternating halves, so one barrier per call is enough).
template <int kTeam> __device__ __forceinline__ float team_sum(float v, float (*red)[32], int& flip) {
#pragma unroll
  for (int o = (kTeam < 32 ? kTeam : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (kTeam > 32) {
    constexpr int kWarps = kTeam / 32;
    const int warp = threadIdx.x / 32, first = warp / kWarps * kWarps;
    if (threadIdx.x % 32 == 0) red[flip][warp] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll 8
    for (int w = 0; w < kWarps; ++w) v += red[flip][first + w];
    flip ^= 1;
  }
  return v;
}
template <int kTeam> __device__ __forceinline__ float2 team_sum(float2 v, float2 (*red)[32], int& flip) {
#pragma unroll
  for (int o = (kTeam < 32 ? kTeam : 32) / 2; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if constexpr (kTeam > 32) {
    constexpr int kWarps = kTeam / 32;
    const int warp = threadIdx.x / 32, first = warp / kWarps * kWarps;
    if (threadIdx.x % 32 == 0) red[flip][warp] = v;
    __syncthreads();
    v = make_float2(0.f, 0.f);
#pragma unroll 8
    for (int w = 0; w < kWarps; ++w) v = __fadd2_rn(v, red[flip][first + w]);
    flip ^= 1;
  }
  return v;
}

template <int kTeam> constexpr int block_threads() { return kTeam > kBlock ? kTeam : kBlock; }

// The rows of a block: of group blockIdx.x (neighbouring blocks take neighbouring memory) the rows n = cls + classes k, k = this team's first, then every `step`
// further; all start `shift` elements behind a 16-byte boundary.
template <int kVec, int kTeams> struct Rows {
  int groups, g, classes, cls, shift;
  long long n_rows, first, step;
  __device__ Rows(long long n_rows_, int groups_, int d, int team) : groups(groups_), g(blockIdx.x), n_rows(n_rows_) {
    classes = d % kVec ? kVec : 1;
    cls = blockIdx.y % classes;
    const int part = blockIdx.y / classes, parts = gridDim.y / classes;
    shift = (int)(((long long)cls * groups + g) % kVec * (d % kVec) % kVec);
    first = (long long)part * kTeams + team;
    step = (long long)parts * kTeams;
  }
  __device__ long long n(long long k) const { return cls + classes * k; }
  // team-independent bound: whether any team of the block has a row at its k-th step
  __device__ bool any(long long k, int team) const { return n(k - team) < n_rows; }
};

// kNV vectors per thread: columns (i kTeam + lane) kVec - shift + e.  kExact: the team's vectors are the row, no more.
template <typename T, int kTeam, int kNV, bool kExact>
__global__ void __launch_bounds__(block_threads<kTeam>())
    k_layer_norm(const T* __restrict__ x, const float* __restrict__ weight, const float* __restrict__ bias,
                 long long n_rows, int groups, int d, float eps, T* __restrict__ y, float* __restrict__ mean,
                 float* __restrict__ rstd) {
  constexpr int kVec = kVecOf<T>, kPairs = kVec / 2, kTeams = block_threads<kTeam>() / kTeam;
  __shared__ float red[2][32];
  int flip = 0;
  const int lane = threadIdx.x % kTeam, team = threadIdx.x / kTeam;
  const Rows<kVec, kTeams> rows(n_rows, groups, d, team);
  const int shift = kExact ? 0 : rows.shift;
  const float inv_d = 1.f / (float)d;
  const long long total = n_rows * groups * d;
  float2 w[kNV][kPairs], bi[kNV][kPairs];
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    const int c = (i * kTeam + lane) * kVec - shift;
    load_par<kVec>(weight ? weight + (long long)rows.g * d : nullptr, c, d, 1.f, w[i]);
    load_par<kVec>(bias ? bias + (long long)rows.g * d : nullptr, c, d, 0.f, bi[i]);
  }
  auto load = [&](long long k, uint4 (&raw)[kNV]) {
    const long long n = rows.n(k), at = (n * groups + rows.g) * d;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * kTeam + lane) * kVec - shift;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (n < n_rows) {
        if (kExact) raw[i] = *reinterpret_cast<const uint4*>(x + at + c);
        else if (c < d) raw[i] = load_cols(x, at, c, d, total);
      }
    }
  };
  auto prefetch = [&](long long k) {
    const long long n = rows.n(k), at = (n * groups + rows.g) * d;
    if (n < n_rows && lane % 8 == 0)
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kTeam + lane) * kVec - shift;
        if (kExact || c < d) prefetch_line(x + at + c);
      }
  };
  uint4 next[kNV];
  load(rows.first, next);
  prefetch(rows.first + rows.step);
  for (long long k = rows.first; rows.any(k, team); k += rows.step) {
    float2 v[kNV][kPairs];
#pragma unroll
    for (int i = 0; i < kNV; ++i)
      unpack<T>(kExact ? next[i] : clear_outside<T>(next[i], (i * kTeam + lane) * kVec - shift, d), v[i]);
    load(k + rows.step, next);
    prefetch(k + kAhead * rows.step);
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int e = 0; e < kPairs; ++e)
        s2 = __fadd2_rn(s2, v[i][e]);
    // Divided, not times 1 / d: where the sum is exact (a constant row of few digits) so is the mean, at any width, and
    // the centred row is zero instead of the mean's rounding times a large rstd.  kExact has a power of two for d,
    // where the product is the quotient (the division costs 1.5 % there: 48360 x 24 rows of 128).
    const float sum = team_sum<kTeam>(s2.x + s2.y, red, flip), mu = kExact ? sum * inv_d : sum / (float)d;
    s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * kTeam + lane) * kVec - shift;
#pragma unroll
      for (int e = 0; e < kPairs; ++e) v[i][e] = __fadd2_rn(v[i][e], both(-mu));
      if (!kExact && (c < 0 || c + kVec > d))
#pragma unroll
        for (int e = 0; e < kPairs; ++e) v[i][e] = inside(v[i][e], c + 2 * e, d);
#pragma unroll
      for (int e = 0; e < kPairs; ++e) s2 = __ffma2_rn(v[i][e], v[i][e], s2);
    }
    const float r = rsqrtf(team_sum<kTeam>(s2.x + s2.y, red, flip) * inv_d + eps);
    const long long n = rows.n(k), row = n * groups + rows.g;
    if (n >= n_rows) continue;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * kTeam + lane) * kVec - shift;
#pragma unroll
      for (int e = 0; e < kPairs; ++e) v[i][e] = __ffma2_rn(__fmul2_rn(v[i][e], both(r)), w[i][e], bi[i][e]);
      if (kExact) *reinterpret_cast<uint4*>(y + row * d + c) = pack<T>(v[i]);
      else if (c < d) store_cols(y, row * d, c, d, v[i]);
    }
    if (lane == 0) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = r;
    }
  }
}

template <typename T, int kTeam, int kNV, bool kExact>
__global__ void __launch_bounds__(block_threads<kTeam>(), kTeam > kBlock ? 1 : 2)
    k_layer_norm_grad(const T* __restrict__ x, const T* __restrict__ dy, const float* __restrict__ weight,
                      const float* __restrict__ mean, const float* __restrict__ rstd, long long n_rows, int groups,
                      int d, T* __restrict__ dx, float* __restrict__ part) {
  constexpr int kVec = kVecOf<T>, kPairs = kVec / 2, kTeams = block_threads<kTeam>() / kTeam;
  __shared__ float2 red[2][32];
  int flip = 0;
  const int lane = threadIdx.x % kTeam, team = threadIdx.x / kTeam;
  const Rows<kVec, kTeams> rows(n_rows, groups, d, team);
  const int shift = kExact ? 0 : rows.shift;
  const float inv_d = 1.f / (float)d;
  const long long total = n_rows * groups * d;
  float2 w[kNV][kPairs], dw[kNV][kPairs], db[kNV][kPairs];
#pragma unroll
  for (int i = 0; i < kNV; ++i) {
    load_par<kVec>(weight ? weight + (long long)rows.g * d : nullptr, (i * kTeam + lane) * kVec - shift, d, 1.f, w[i]);
#pragma unroll
    for (int e = 0; e < kPairs; ++e) dw[i][e] = db[i][e] = make_float2(0.f, 0.f);
  }
  struct Row {
    uint4 x[kNV], g[kNV];
    float mu, r;
  };
  auto load = [&](long long k, Row& q) {
    const long long n = rows.n(k), row = n * groups + rows.g;
    const bool live = n < n_rows;
    q.mu = live ? mean[row] : 0.f;
    q.r = live ? rstd[row] : 0.f;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * kTeam + lane) * kVec - shift;
      q.x[i] = q.g[i] = make_uint4(0, 0, 0, 0);
      if (live) {
        if (kExact) {
          q.x[i] = *reinterpret_cast<const uint4*>(x + row * d + c);
          q.g[i] = *reinterpret_cast<const uint4*>(dy + row * d + c);
        } else if (c < d) {
          q.x[i] = load_cols(x, row * d, c, d, total);
          q.g[i] = load_cols(dy, row * d, c, d, total);
        }
      }
    }
  };
  auto prefetch = [&](long long k) {
    const long long n = rows.n(k), at = (n * groups + rows.g) * d;
    if (n < n_rows && lane % 8 == 0)
#pragma unroll
      for (int i = 0; i < kNV; ++i) {
        const int c = (i * kTeam + lane) * kVec - shift;
        if (kExact || c < d) {
          prefetch_line(x + at + c);
          prefetch_line(dy + at + c);
        }
      }
  };
  Row next;
  load(rows.first, next);
  prefetch(rows.first + rows.step);
  for (long long k = rows.first; rows.any(k, team); k += rows.step) {
    float2 xc[kNV][kPairs], g[kNV][kPairs];
    const float r = next.r, mu = next.mu;
    float2 s = make_float2(0.f, 0.f), s2 = s;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * kTeam + lane) * kVec - shift;
      unpack<T>(kExact ? next.x[i] : clear_outside<T>(next.x[i], c, d), xc[i]);
      unpack<T>(kExact ? next.g[i] : clear_outside<T>(next.g[i], c, d), g[i]);
#pragma unroll
      for (int e = 0; e < kPairs; ++e) {
        // xh = (x - mu) r is not formed: r goes to dy here, to the row's sum and to dx below.  The difference comes first,
        // where a far mean cancels.  Outside the row dy is zero, and x - mu = -mu is finite, as -mu r need not be
        // (zero times that would be NaN).
        xc[i][e] = __fadd2_rn(xc[i][e], both(-mu));
        dw[i][e] = __ffma2_rn(__fmul2_rn(g[i][e], both(r)), xc[i][e], dw[i][e]);
        db[i][e] = __fadd2_rn(db[i][e], g[i][e]);
        g[i][e] = __fmul2_rn(g[i][e], w[i][e]);
        s = __fadd2_rn(s, g[i][e]);
        s2 = __ffma2_rn(g[i][e], xc[i][e], s2);
      }
    }
    load(k + rows.step, next);
    prefetch(k + kAhead * rows.step);
    const float2 c12 = team_sum<kTeam>(make_float2(s.x + s.y, s2.x + s2.y), red, flip);
    const float c1 = -c12.x * inv_d, c2 = -(c12.y * r) * (r * inv_d);
    const long long n = rows.n(k), row = n * groups + rows.g;
    if (n >= n_rows) continue;
#pragma unroll
    for (int i = 0; i < kNV; ++i) {
      const int c = (i * kTeam + lane) * kVec - shift;
#pragma unroll
      for (int e = 0; e < kPairs; ++e)
        g[i][e] = __fmul2_rn(__ffma2_rn(xc[i][e], both(c2), __fadd2_rn(g[i][e], both(c1))), both(r));
      if (kExact) *reinterpret_cast<uint4*>(dx + row * d + c) = pack<T>(g[i]);
      else if (c < d) store_cols(dx, row * d, c, d, g[i]);
    }
  }
  if (!part) return;
  // the block's teams, then the partial sums [2][gridDim.y][groups][d]
  float* pw = part + ((long long)blockIdx.y * groups + rows.g) * d;
  float* pb = pw + (long long)gridDim.y * groups * d;
  if constexpr (kTeams == 1) {
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const int c = (i * kTeam + lane) * kVec - shift + e;
        if (c >= 0 && c < d) {
          pw[c] = e & 1 ? dw[i][e / 2].y : dw[i][e / 2].x;
          pb[c] = e & 1 ? db[i][e / 2].y : db[i][e / 2].x;
        }
      }
  } else {
    __shared__ float acc[block_threads<kTeam>()][kVec + 1];   // + 1: one column's teams on separate banks
#pragma unroll
    for (int i = 0; i < kNV; ++i)
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float2 q = which ? db[i][e / 2] : dw[i][e / 2];
          acc[threadIdx.x][e] = e & 1 ? q.y : q.x;
        }
        __syncthreads();
        for (int j = threadIdx.x; j < kTeam * kVec; j += block_threads<kTeam>()) {
          const int c = i * kTeam * kVec + j - shift;
          if (c >= 0 && c < d) {
            float t = 0.f;
#pragma unroll 8
            for (int m = 0; m < kTeams; ++m) t += acc[m * kTeam + j / kVec][j % kVec];
            (which ? pb : pw)[c] = t;
          }
        }
      }
  }
}

// sums of `parts` partial rows: 32 columns per block, 32 threads per column, then a fixed tree
__global__ void __launch_bounds__(1024) k_norm_sum(const float* __restrict__ part, int parts, int cols,
                                                   float* __restrict__ dweight, float* __restrict__ dbias) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float* dst = blockIdx.y ? dbias : dweight;
  if (!dst) return;
  part += (long long)blockIdx.y * parts * cols;
  float t = 0.f;
  if (c < cols)
#pragma unroll 8
    for (int p = warp; p < parts; p += 32) t += part[(long long)p * cols + c];
  acc[warp][lane] = t;
  __syncthreads();
  t = warp_sum(acc[lane][warp]);              // thread (warp, lane): column `warp`, part sums of all warps
  if (lane == 0 && blockIdx.x * 32 + warp < cols) dst[blockIdx.x * 32 + warp] = t;
}

// The team and the vectors per thread for a row of `vecs` vectors: two vectors (fp32: four) per thread, and the
// smallest power of two of threads.
template <typename T> constexpr int kNVOf = 8 / kVecOf<T> * 2;
struct NormShape {
  int team, nv;
  bool exact;
};
template <typename T> NormShape norm_shape(int d) {
  const int vecs = d / kVecOf<T> + (d % kVecOf<T> ? 2 : 0);       // a shift may open one vector more
  for (int team = 1; team <= 1024; team *= 2)
    if (vecs <= kNVOf<T> * team) return {team, kNVOf<T>, d == team * kNVOf<T> * kVecOf<T>};
  return {1024, kNVOf<T> + 1, false};
}
template <template <typename, int, int, bool> class Op, typename T, bool kExact, typename A>
cudaError_t by_team(int team, const A& a) {
  constexpr int kNV = kNVOf<T>;
  switch (team) {
    case 1: return Op<T, 1, kNV, kExact>::run(a);
    case 2: return Op<T, 2, kNV, kExact>::run(a);
    case 4: return Op<T, 4, kNV, kExact>::run(a);
    case 8: return Op<T, 8, kNV, kExact>::run(a);
    case 16: return Op<T, 16, kNV, kExact>::run(a);
    case 32: return Op<T, 32, kNV, kExact>::run(a);
    case 64: return Op<T, 64, kNV, kExact>::run(a);
    case 128: return Op<T, 128, kNV, kExact>::run(a);
    case 256: return Op<T, 256, kNV, kExact>::run(a);
    case 512: return Op<T, 512, kNV, kExact>::run(a);
    default: return Op<T, 1024, kNV, kExact>::run(a);
  }
}
template <template <typename, int, int, bool> class Op, typename T, typename A> cudaError_t by_width(const A& a) {
  const NormShape s = norm_shape<T>(a.d);
  if (s.nv > kNVOf<T>) return Op<T, 1024, kNVOf<T> + 1, false>::run(a);
  return s.exact ? by_team<Op, T, true>(s.team, a) : by_team<Op, T, false>(s.team, a);
}

// Blocks per group: `threads` per SM over all groups, and no more than have a row; a multiple of the classes of rows
// (at least one block each).  Every block reads its parameters first, and in the backward leaves a partial sum.
// Long rows (teams of a warp or more): two blocks, which run at once; with four, the backward takes 16 % longer for
// 4032 rows of 1999 and 17 % for 3000 of 8192.  Short rows, whose parameters are short: several times that, so that
// the last blocks end together (48360 x 24 rows of 128: backward 12 % less with 12 blocks than with four, forward 6 % less
// with 24 than with eight; inputs in turn), but a third of it where rows start at odd places and parameters are read
// one by one (100000 rows of 77: 28 % less).
struct NormThreads {
  int long_rows, short_rows, short_odd;
};
constexpr NormThreads kForwardThreads = {2 * kBlock, 24 * kBlock, 8 * kBlock},
                      kGradThreads = {2 * kBlock, 12 * kBlock, 4 * kBlock};
int norm_parts(long long rows, int groups, int d, int dtype, const NormThreads& t) {
  const int vec = dtype == VDN_DTYPE_BF16 ? 8 : 4, classes = d % vec ? vec : 1;
  const int team = (dtype == VDN_DTYPE_BF16 ? norm_shape<__nv_bfloat16>(d) : norm_shape<float>(d)).team;
  const int block = team > kBlock ? team : kBlock, teams = block / team;
  const long long per_class = (rows / groups + classes - 1) / classes, most = (per_class + teams - 1) / teams;
  const int threads = team >= 32 ? t.long_rows : classes == 1 ? t.short_rows : t.short_odd;
  const long long blocks = 148LL * threads / block, all = (long long)groups * classes;
  const long long want = (blocks + all - 1) / all;
  return (int)(want < most ? want : most) * classes;
}

struct NormArgs {
  const void *x, *dy;
  const float *weight, *bias;
  float *mean, *rstd;
  const float *mean_in, *rstd_in;
  long long rows;        // of d elements
  int groups, d;
  float eps;
  void* out;
  float* part;
  int parts;
  cudaStream_t stream;
};

template <typename T, int kTeam, int kNV, bool kExact> struct Forward {
  static cudaError_t run(const NormArgs& a) {
    k_layer_norm<T, kTeam, kNV, kExact><<<dim3((unsigned)a.groups, (unsigned)a.parts), block_threads<kTeam>(), 0, a.stream>>>(
        (const T*)a.x, a.weight, a.bias, a.rows / a.groups, a.groups, a.d, a.eps, (T*)a.out, a.mean, a.rstd);
    return cudaGetLastError();
  }
};
template <typename T, int kTeam, int kNV, bool kExact> struct Backward {
  static cudaError_t run(const NormArgs& a) {
    k_layer_norm_grad<T, kTeam, kNV, kExact>
        <<<dim3((unsigned)a.groups, (unsigned)a.parts), block_threads<kTeam>(), 0, a.stream>>>(
            (const T*)a.x, (const T*)a.dy, a.weight, a.mean_in, a.rstd_in, a.rows / a.groups, a.groups, a.d, (T*)a.out,
            a.part);
    return cudaGetLastError();
  }
};

template <template <typename, int, int, bool> class Op> cudaError_t launch_norm(int dtype, const NormArgs& a) {
  return dtype == VDN_DTYPE_BF16 ? by_width<Op, __nv_bfloat16>(a) : by_width<Op, float>(a);
}

vdn_status norm_args(long long rows, int groups, int d, int dtype) {
  if (rows < 1 || groups < 1 || d < 1 || rows % groups) return VDN_ERR_INVALID_ARG;
  if (dtype != VDN_DTYPE_F32 && dtype != VDN_DTYPE_BF16) return VDN_ERR_INVALID_ARG;
  if (d > kNormMaxWidth || groups > 65535 || rows > 0x7fffffffLL || (long long)groups * d > (1 << 28))
    return VDN_ERR_UNSUPPORTED;
  return VDN_OK;
}

size_t norm_bytes(long long rows, int d, int dtype) { return (size_t)rows * d * (dtype == VDN_DTYPE_BF16 ? 2 : 4); }

}  // namespace
}  // namespace vdn

using namespace vdn;

extern "C" {

size_t vdn_layer_norm_backward_workspace_size(long long rows, int groups, int d, int dtype) {
  if (norm_args(rows, groups, d, dtype) != VDN_OK) return 0;
  const size_t n = (size_t)2 * norm_parts(rows, groups, d, dtype, kGradThreads) * groups * d * sizeof(float);
  return (n + 255) & ~(size_t)255;
}

vdn_status vdn_layer_norm_forward(const void* x, const float* weight, const float* bias, long long rows, int groups,
                                  int d, int dtype, float eps, void* y, float* mean, float* rstd, void* stream) {
  vdn_status st = norm_args(rows, groups, d, dtype);
  if (st != VDN_OK) return st;
  if (!x || !y || !std::isfinite(eps) || eps < 0.f) return VDN_ERR_INVALID_ARG;
  const size_t big = norm_bytes(rows, d, dtype), par = (size_t)groups * d * 4;
  Buffers buf;
  buf.in(x, big);
  buf.in(weight, par);
  buf.in(bias, par);
  buf.out(y, big);
  buf.out(mean, (size_t)rows * 4);
  buf.out(rstd, (size_t)rows * 4);
  if ((st = buf.check()) != VDN_OK) return st;
  NormArgs a{};
  a.x = x; a.weight = weight; a.bias = bias;
  a.rows = rows; a.groups = groups; a.d = d;
  a.eps = eps;
  a.out = y; a.mean = mean; a.rstd = rstd;
  a.parts = norm_parts(rows, groups, d, dtype, kForwardThreads);
  a.stream = (cudaStream_t)stream;
  return launch_norm<Forward>(dtype, a) == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
}

vdn_status vdn_layer_norm_backward(const void* x, const void* dy, const float* mean, const float* rstd,
                                   const float* weight, long long rows, int groups, int d, int dtype, void* workspace,
                                   size_t workspace_bytes, void* dx, float* dweight, float* dbias, void* stream) {
  vdn_status st = norm_args(rows, groups, d, dtype);
  if (st != VDN_OK) return st;
  if (!x || !dy || !mean || !rstd || !dx) return VDN_ERR_INVALID_ARG;
  const bool sums = dweight || dbias;
  if (sums && !workspace) return VDN_ERR_INVALID_ARG;
  const size_t big = norm_bytes(rows, d, dtype), par = (size_t)groups * d * 4;
  const size_t need = vdn_layer_norm_backward_workspace_size(rows, groups, d, dtype);
  Buffers buf;
  buf.in(x, big);
  buf.in(dy, big);
  buf.in(mean, (size_t)rows * 4);
  buf.in(rstd, (size_t)rows * 4);
  buf.in(weight, par);
  buf.out(dx, big);
  buf.out(dweight, par);
  buf.out(dbias, par);
  if (sums) buf.workspace(workspace, need);
  if ((st = buf.check()) != VDN_OK) return st;
  if (sums && workspace_bytes < need) return VDN_ERR_WORKSPACE;
  NormArgs a{};
  a.x = x; a.dy = dy; a.weight = weight;
  a.mean_in = mean; a.rstd_in = rstd;
  a.rows = rows; a.groups = groups; a.d = d;
  a.out = dx;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  a.parts = norm_parts(rows, groups, d, dtype, kGradThreads);
  a.stream = (cudaStream_t)stream;
  cudaError_t e = launch_norm<Backward>(dtype, a);
  if (e == cudaSuccess && sums) {
    const int cols = groups * d;
    k_norm_sum<<<dim3((unsigned)((cols + 31) / 32), 2), 1024, 0, a.stream>>>(a.part, a.parts, cols, dweight, dbias);
    e = cudaGetLastError();
  }
  return e == cudaSuccess ? VDN_OK : VDN_ERR_CUDA;
}

}  // extern "C"
