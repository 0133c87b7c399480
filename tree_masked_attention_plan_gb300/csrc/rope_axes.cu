// Rotary positions with several axes (an image patch's time, height and width; a text token has
// the same position on all of them): rotate-half RoPE whose frequency c turns by the position on
// the axis that c belongs to.
//   x'_c = x_c cos(a) - x_{c+d/2} sin(a),  x'_{c+d/2} = x_{c+d/2} cos(a) + x_c sin(a),
//   a = pos[axis(c)][t] * theta^(-2c/d);   the gradient goes through the rotation by -a.
// Angles are exact to fp32 at any int32 position: a frequency is held as a 64-bit fraction of a
// turn, so that pos * frequency wraps modulo one turn by itself in integer arithmetic, and only
// the wrapped fraction becomes a float (error 2^-26 turns, where pos * frequency in fp32 loses
// whole radians beyond position 10^6).  The table is made in pairs of doubles: in doubles alone its frequencies were
// off by up to 2^-55, 2^-24 turns at position 2^31, and for theta < 1, where they are many turns, by far more.
// HBM-bound: every head of q and k is read and written once.  32768 tokens of 40 heads of 128: 104 us, 6.4 TB/s;
// the gradient of 9973 tokens of 32 heads of 64: 16.5 us, 5.0 TB/s (82 MB, of which much stays in L2).
#include <cmath>

#include "common.cuh"

namespace ta {
namespace {

constexpr int kAxesThreads = 256;

struct AxesTable {
  uint64_t turn[64];       // theta^(-2c/d) / (2 pi) as a fraction of 2^64
  uint8_t axis[64];
};

// A warp rotates all heads of one token (or its share of them): HD/16 lanes cover a head's row,
// eight frequencies a lane, so a lane's sines are computed once and serve every head it visits.
template <int HD>
__global__ void __launch_bounds__(kAxesThreads) k_rope_axes(const __grid_constant__ AxesTable tab,
                                                            const int32_t* __restrict__ pos, int N, int split,
                                                            float sign, const uint4* q, uint4* qr, int Hq,
                                                            const uint4* k, uint4* kr, int Hkv) {
  constexpr int VPR = HD / 16;                    // lanes per head: 16-byte vectors per half row
  constexpr int ROWS = 32 / VPR;                  // heads a warp rotates at once
  const int64_t wid = (int64_t)blockIdx.x * (kAxesThreads / 32) + (threadIdx.x >> 5);
  const int t = static_cast<int>(wid / split), part = static_cast<int>(wid % split);
  if (t >= N) return;
  const int v = threadIdx.x % VPR, row0 = (threadIdx.x & 31) / VPR;
  float cs[8], sn[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = 8 * v + e;
    const int64_t p = pos[(size_t)tab.axis[c] * N + t];
    const uint64_t phase = static_cast<uint64_t>(p) * tab.turn[c];
    const int32_t frac = static_cast<int32_t>(phase >> 32);          // [-1/2, 1/2) turn
    sincospif(static_cast<float>(frac) * 0x1p-31f, &sn[e], &cs[e]);
    sn[e] *= sign;
  }
  const int H = Hq + Hkv;
  for (int h = part * ROWS + row0; h < H; h += split * ROWS) {
    const bool isq = h < Hq;
    const uint4* src = isq ? q : k;
    uint4* dst = isq ? qr : kr;
    const size_t row = isq ? (size_t)t * Hq + h : (size_t)t * Hkv + (h - Hq);
    const size_t at = row * (HD / 8) + v;
    const uint4 a = src[at], b = src[at + VPR];
    const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
    uint32_t oa[4], ob[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float xl = bf16lo(av[e]), xh = bf16hi(av[e]), yl = bf16lo(bv[e]), yh = bf16hi(bv[e]);
      oa[e] = pack_bf16(xl * cs[2 * e] - yl * sn[2 * e], xh * cs[2 * e + 1] - yh * sn[2 * e + 1]);
      ob[e] = pack_bf16(yl * cs[2 * e] + xl * sn[2 * e], yh * cs[2 * e + 1] + xh * sn[2 * e + 1]);
    }
    dst[at] = make_uint4(oa[0], oa[1], oa[2], oa[3]);
    dst[at + VPR] = make_uint4(ob[0], ob[1], ob[2], ob[3]);
  }
}

// A number as the sum of two doubles, about 106 bits.  Dekker's and Knuth's error-free sums, products through fma.
struct Pair {
  double hi, lo;
};
Pair pair_of(double a, double b) {                   // |a| >= |b|
  const double s = a + b;
  return {s, b - (s - a)};
}
Pair times(Pair a, Pair b) {
  const double p = a.hi * b.hi, e = std::fma(a.hi, b.hi, -p);
  return pair_of(p, e + std::fma(a.hi, b.lo, a.lo * b.hi));
}
Pair root(Pair a) {                                  // one Newton step from the double's root
  const double s = std::sqrt(a.hi), d = std::fma(-s, s, a.hi) + a.lo;
  return pair_of(s, d / (2.0 * s));
}
Pair inverse(Pair a) {
  const double q = 1.0 / a.hi, r = std::fma(-q, a.hi, 1.0) - q * a.lo;
  return pair_of(q, q * r);
}
// theta^(-c / half) / (2 pi) turns for c < half, as fractions of 2^64; half is a power of two.  The powers of one root
// (two chains, each other's latency): their error grows to some 2^-97 of their size; whole turns (theta < 1) drop out.
void turns_of(double theta, int half, uint64_t* turn) {
  Pair r{theta, 0.0};
  for (int h = half; h > 1; h /= 2) r = root(r);
  r = inverse(r);
  const Pair start{0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};        // 1 / (2 pi)
  Pair f[2] = {start, times(start, r)};
  r = times(r, r);
  for (int c = 0; c < half; ++c) {
    Pair& g = f[c & 1];
    const double hi = g.hi - std::floor(g.hi), lo = g.lo - std::floor(g.lo + 0.5);       // [0, 1), [-1/2, 1/2)
    turn[c] = static_cast<uint64_t>(hi * 0x1p64) + static_cast<uint64_t>(static_cast<int64_t>(lo * 0x1p64));
    g = times(g, r);
  }
}

// The axis of every frequency.  In runs: the first sections[0] frequencies on axis 0, and so on.
// Interleaved: axis i >= 1 takes frequencies i, i + n, i + 2n, ... until it has sections[i] of
// them; the rest belongs to axis 0.  False where the sections do not describe d/2 frequencies.
bool axes_of(const int32_t* sections, int n, int interleaved, int half, uint8_t* axis) {
  int64_t sum = 0;
  for (int i = 0; i < n; ++i) {
    if (sections[i] < 0) return false;
    sum += sections[i];
  }
  if (sum != half) return false;
  if (!interleaved) {
    int c = 0;
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < sections[i]; ++j) axis[c++] = static_cast<uint8_t>(i);
    return true;
  }
  for (int c = 0; c < half; ++c) axis[c] = 0;
  for (int i = 1; i < n; ++i)
    for (int j = 0; j < sections[i]; ++j) {
      const int c = i + n * j;
      if (c >= half) return false;
      axis[c] = static_cast<uint8_t>(i);
    }
  return true;
}

int rope_axes(const tree_plan_t* plan, const int32_t* pos, const int32_t* sections, int n_axes, int interleaved,
              const tree_bf16* q, const tree_bf16* k, tree_bf16* qr, tree_bf16* kr, int Hq, int Hkv, int d,
              float theta, float sign, tree_stream_t stream) {
  int rc = plan_ok(plan);
  if (rc) return rc;
  if (!pos || !sections || !q || !k || !qr || !kr) return TREE_ERR_ARG;
  if ((d != 64 && d != 128) || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || !(theta > 0.f) || !std::isfinite(theta) ||
      n_axes < 1 || n_axes > TREE_MAX_AXES)
    return TREE_ERR_SHAPE;
  for (const void* p : {(const void*)q, (const void*)k, (const void*)qr, (const void*)kr})
    if (reinterpret_cast<uintptr_t>(p) & 15) return TREE_ERR_ARG;
  if (reinterpret_cast<uintptr_t>(pos) & 3) return TREE_ERR_ARG;
  AxesTable tab;
  const int half = d / 2;
  if (!axes_of(sections, n_axes, interleaved, half, tab.axis)) return TREE_ERR_SHAPE;
  // A row is read before it is written, by the same lanes: an output may be its own input, but touch nothing else.
  const size_t row = (size_t)plan->n_tokens * d * 2, nq = row * Hq, nk = row * Hkv, np = (size_t)plan->n_tokens * n_axes * 4;
  if (buffers_meet(qr, nq, kr, nk) || buffers_meet(qr, nq, k, nk) || buffers_meet(kr, nk, q, nq) ||
      buffers_meet(qr, nq, pos, np) || buffers_meet(kr, nk, pos, np) || (qr != q && buffers_meet(qr, nq, q, nq)) ||
      (kr != k && buffers_meet(kr, nk, k, nk)))
    return TREE_ERR_ARG;
  turns_of(theta, half, tab.turn);
  rc = check_device();
  if (rc) return rc;
  const int N = plan->n_tokens;
  const int rows = d == 128 ? 4 : 8;
  // One warp a token once there are enough of them to fill the GPU; with few tokens a token's
  // heads are dealt to several warps (48 tokens of 40 heads: ten warps each, 2.6 us instead of 5.5).
  const int most = (Hq + Hkv + rows - 1) / rows;
  int split = 1;
  while (split < most && (int64_t)N * split < 152 * 16) ++split;
  const int64_t warps = (int64_t)N * split;
  const unsigned blocks = (unsigned)((warps + kAxesThreads / 32 - 1) / (kAxesThreads / 32));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (d == 128)
    k_rope_axes<128><<<blocks, kAxesThreads, 0, s>>>(tab, pos, N, split, sign, (const uint4*)q, (uint4*)qr, Hq,
                                                     (const uint4*)k, (uint4*)kr, Hkv);
  else
    k_rope_axes<64><<<blocks, kAxesThreads, 0, s>>>(tab, pos, N, split, sign, (const uint4*)q, (uint4*)qr, Hq,
                                                    (const uint4*)k, (uint4*)kr, Hkv);
  return record_cuda(cudaGetLastError());
}

}  // namespace
}  // namespace ta

using namespace ta;

extern "C" {

int tree_rope_axes_fwd(const tree_plan_t* plan, const int32_t* pos, const int32_t* sections, int n_axes,
                       int interleaved, const tree_bf16* q, const tree_bf16* k, tree_bf16* qr, tree_bf16* kr, int Hq,
                       int Hkv, int d, float theta, tree_stream_t stream) {
  return rope_axes(plan, pos, sections, n_axes, interleaved, q, k, qr, kr, Hq, Hkv, d, theta, 1.f, stream);
}

int tree_rope_axes_bwd(const tree_plan_t* plan, const int32_t* pos, const int32_t* sections, int n_axes,
                       int interleaved, const tree_bf16* dqr, const tree_bf16* dkr, tree_bf16* dq, tree_bf16* dk,
                       int Hq, int Hkv, int d, float theta, tree_stream_t stream) {
  return rope_axes(plan, pos, sections, n_axes, interleaved, dqr, dkr, dq, dk, Hq, Hkv, d, theta, -1.f, stream);
}

}  // extern "C"
