// Gated linear recurrence along the root paths of a packed tree ("Tree Training 技术详解", section
// 9.1: a recurrent layer's node starts from its parent's final state, h_c(0) = h_parent(end)):
//   h_t = a_t h_prev(t) + b_t,   y_t = h_t,
//   sigmoid gate: a = sigmoid(g), b = (1 - a) x;      log gate: a = exp(min(g, 0)), b = x,
// prev(t) the token before t on its root path, per channel.  Its gradient, from the leaves up:
//   lam_t = dy_t + sum_{s: prev(s) = t} a_s lam_s,
//   sigmoid: dx = (1 - a) lam, dg = a (1 - a) (h_prev - x) lam;   log: dx = lam, dg = a h_prev lam.
// In depth-first packing prev(t) is t - 1 but for the first token of a root and of every child
// after the first: those tokens are the breaks of the packed sequence, and a break starts from the
// final state of a node that lies before it.
//
// HBM-bound: the forward reads g and x and writes y once, the backward reads g, x, dy and writes
// dg, dx once.  A unit of work is a tile of 128 tokens by 128 bytes of channels.  A step of the
// recurrence is the map h -> a h + b, and maps compose, so a tile needs its neighbours for one
// value per channel only: it adds its own 128 steps up to one map, publishes that, takes the state
// before it from the maps of the tiles before it, and then knows every h.  Tiles are handed out
// in packed order (the backward: from the end) by a counter, so that whatever a tile waits for is
// done or being worked on, however few blocks the GPU runs at a time; every wait has a limit.
// The order in which states and maps are joined depends on the tree alone: the result does not
// change from run to run.
//
// Precision: states, gates and gradients are fp32.  A decay close to one is held as what it
// lacks to one: p = -(1 - a) where a > 1/2, p = a elsewhere, so that a memory of thousands of
// tokens does not lose its length to the rounding of a; the step h + (p h + b) then adds a small
// increment to h.
#include <algorithm>
#include <atomic>

#include "common.cuh"

namespace ta {
int make_tmap_bf16_2d(CUtensorMap* m, const void* base, int inner, int rows, int box_inner, int box_rows);  // host.cu

namespace {

constexpr int kScanWarps = 8;               // warps that share a tile: 16 tokens each
constexpr int kFwdGroups = 2, kBwdGroups = 1;      // groups of mapping warps, which take tiles in turn
constexpr int kEnds = 2;                            // tiles past the last that the loading warp announces as ends
constexpr int kJoiners = 2;                         // joining warps, which take tiles in turn
// a block: the mapping warps, the walking warps, one that loads, one that publishes, the joining ones
constexpr int scan_threads(int groups) { return 32 * ((groups + 1) * kScanWarps + 2 + kJoiners); }
constexpr int kWarpTokens = TILE / kScanWarps;
constexpr int kRow = 128;                   // bytes of a tile's row: 64 bf16 or 32 fp32 channels, a word a lane
constexpr int kPlane = TILE * kRow;         // one tensor's rows of a tile
constexpr int kScanGroup = 8;               // at most this many maps are joined to a state

constexpr int kLinkChain = -1;             // the token before on the path is the one before in packed order
constexpr int kLinkRoot = -2;              // the token starts from its node's initial state

struct ScanTree {
  const int32_t* tok_node;
  const int32_t* tok_start;
  const int32_t* sub_end;
  const int32_t* parent;
  const int32_t* node_len;
  int N, n_nodes, n_tiles;
};

// What the kernels keep in the workspace.  Per packed token:
//   link  kLinkChain, kLinkRoot, or the node whose final state the token starts from (a break)
//   end   the token's node if it is the node's last token, else -1
//   kid   for a node's last token: the second of the nodes that start from it (the first one is its
//         successor in packed order), -1 if there is none
//   sib   for a break: the next node after its own that starts from the same state, -1 if none
// info: per tile, the kInfo bits.  flags: per tile and slab, whether its nodes' rows are written (those
// that breaks start from; backward, those of its breaks).  ctl: the counter that hands out tiles (64
// bits), and a word that stops every wait once one has run out of time.
struct ScanWork {
  int32_t *link, *end, *kid, *sib, *info, *flags, *ctl;
  float *maps, *dnode, *carry;
};

enum : int {
  kInfoBreak = 1,       // holds a break
  kInfoIn = 2,          // its first token follows on the tile before
  kInfoSerial = 4,      // a break starts from a node that ends in this tile
  kInfoEnd = 8,         // holds a node's last token
  kInfoSource = 16,     // holds the last token of a node that a break starts from
  kInfoOut = 32,        // the tile behind follows on its last token
  kInfoSerialBack = 64, // a node's further child, or a break's next sibling, starts in this tile
  kInfoMapped = 128,    // (set by the loading warp) the tile is a plain map of the state before it (gradient behind it)
  kInfoMap = 256,       // (the same) and other tiles join that map
};
// Maps and the states between tiles carry their own arrival: their rows hold this pattern, a NaN that no
// arithmetic gives, until they are written, and whoever needs one polls the value itself.  No flag and no
// fence stands between a tile and the next.
constexpr uint32_t kEmpty = 0xffffffffu;

DEVI int scan_token_ancestor(int v, const ScanTree& t) {
  int a = t.parent[v];
  for (int guard = 0; a >= 0 && a < t.n_nodes && t.node_len[a] == 0 && guard < t.n_nodes; ++guard) a = t.parent[a];
  return (a >= 0 && a < t.n_nodes && t.node_len[a] > 0) ? a : -1;
}

// the link of token j
DEVI int link_of(int j, const ScanTree& t) {
  const int v = t.tok_node[j];
  if (j != t.tok_start[v]) return kLinkChain;
  const int a = scan_token_ancestor(v, t);
  if (a < 0) return kLinkRoot;
  return t.tok_start[a] + t.node_len[a] == j ? kLinkChain : a;
}

// Blocks (tile, share of the channels): links and info, the tile's flags cleared, its map and the state
// behind it marked empty; and the rows that no tile writes are zeroed: those of nodes without tokens, and
// with `inner` of nodes that do not start from nothing.
__global__ void __launch_bounds__(TILE) k_scan_prepare(ScanTree t, ScanWork w, int slabs, int C, int inner,
                                                       float* rows, float* between) {
  __shared__ int bits;
  const int k = blockIdx.x, j = k * TILE + threadIdx.x;
  {
    const uint4 e = make_uint4(kEmpty, kEmpty, kEmpty, kEmpty);
    const int first = blockIdx.y * TILE + threadIdx.x, step = gridDim.y * TILE;
    uint4* m = reinterpret_cast<uint4*>(w.maps + (size_t)k * C * 2);
    uint4* b = reinterpret_cast<uint4*>(between + (size_t)k * C);
    for (int i = first; i < C / 2; i += step) m[i] = e;
    for (int i = first; i < C / 4; i += step) b[i] = e;
    for (int i = first; i < slabs; i += step) w.flags[(size_t)k * slabs + i] = 0;
  }
  if (rows)
    for (int v = k; v < t.n_nodes; v += gridDim.x) {
      if (t.node_len[v] > 0 && !(inner && scan_token_ancestor(v, t) >= 0)) continue;
      for (int c = blockIdx.y * TILE + threadIdx.x; c < C; c += gridDim.y * TILE) rows[(size_t)v * C + c] = 0.f;
    }
  if (blockIdx.y) return;
  if (threadIdx.x == 0) bits = 0;
  if (k == 0 && threadIdx.x < 4) w.ctl[threadIdx.x] = 0;
  __syncthreads();
  if (j < t.N) {
    const int v = t.tok_node[j];
    const int link = link_of(j, t);
    int sib = -1, end = -1, kid = -1, mine = 0;
    if (link != kLinkChain) mine |= kInfoBreak;
    else if (threadIdx.x == 0) mine |= kInfoIn;
    if (link >= 0) {
      if ((t.tok_start[link] + t.node_len[link] - 1) / TILE == k) mine |= kInfoSerial;
      const int next = t.sub_end[v];
      if (next < t.sub_end[link]) {
        sib = t.tok_node[next];
        if (next / TILE == k) mine |= kInfoSerialBack;
      }
    }
    if (j == t.tok_start[v] + t.node_len[v] - 1) {
      end = v;
      mine |= kInfoEnd;
      if (j + 1 < t.sub_end[v]) {
        const int next = t.sub_end[t.tok_node[j + 1]];
        if (next < t.sub_end[v]) {
          kid = t.tok_node[next];
          mine |= kInfoSource;
          if (next / TILE == k) mine |= kInfoSerialBack;
        }
      }
    }
    if (threadIdx.x == TILE - 1 && j + 1 < t.N && link_of(j + 1, t) == kLinkChain) mine |= kInfoOut;
    w.link[j] = link;
    w.end[j] = end;
    w.kid[j] = kid;
    w.sib[j] = sib;
    if (mine) atomicOr(&bits, mine);
  }
  __syncthreads();
  if (threadIdx.x == 0) w.info[k] = bits;
}

// A lane's one or two channels of a value; pairs go through the packed fp32 instructions.
template <int CH>
struct Vec {
  float v[CH];
};
template <int CH>
DEVI Vec<CH> vec(float a) {
  Vec<CH> r;
#pragma unroll
  for (int c = 0; c < CH; ++c) r.v[c] = a;
  return r;
}
DEVI Vec<1> operator+(Vec<1> a, Vec<1> b) { return {{a.v[0] + b.v[0]}}; }
DEVI Vec<1> operator*(Vec<1> a, Vec<1> b) { return {{a.v[0] * b.v[0]}}; }
DEVI Vec<1> vfma(Vec<1> a, Vec<1> b, Vec<1> c) { return {{fmaf(a.v[0], b.v[0], c.v[0])}}; }
DEVI uint64_t f2(Vec<2> a) { return f2_pack(a.v[0], a.v[1]); }
DEVI Vec<2> f2(uint64_t a) {
  Vec<2> r;
  f2_unpack(a, r.v[0], r.v[1]);
  return r;
}
DEVI Vec<2> operator+(Vec<2> a, Vec<2> b) { return f2(f2_add(f2(a), f2(b))); }
DEVI Vec<2> operator*(Vec<2> a, Vec<2> b) { return f2(f2_mul(f2(a), f2(b))); }
DEVI Vec<2> vfma(Vec<2> a, Vec<2> b, Vec<2> c) { return f2(f2_fma(f2(a), f2(b), f2(c))); }
template <int CH>
DEVI Vec<CH> operator-(Vec<CH> a, Vec<CH> b) { return vfma(b, vec<CH>(-1.f), a); }

// A decay a as p: -(1 - a) with the sign bit set where a >= 1/2, a itself elsewhere.  A log gate above zero
// is held at a = 1 and has no gradient: its p is the least negative number, which no other gate gives.
constexpr uint32_t kHeld = 0x80000001u;
DEVI bool near_one(float p) { return __float_as_int(p) < 0; }
template <int CH>
DEVI Vec<CH> pick(Vec<CH> p, Vec<CH> a, Vec<CH> b) {      // a where the decay is near one, else b
#pragma unroll
  for (int c = 0; c < CH; ++c) a.v[c] = near_one(p.v[c]) ? a.v[c] : b.v[c];
  return a;
}
// a h
template <int CH>
DEVI Vec<CH> decayed(Vec<CH> p, Vec<CH> h) { return vfma(p, h, pick(p, h, vec<CH>(0.f))); }
// a h + b.  Sigmoid gate: a h + (1 - a) x is h + p (h - x) or x + p (h - x).
template <int KIND, int CH>
DEVI Vec<CH> advance(Vec<CH> p, Vec<CH> x, Vec<CH> h) {
  if (KIND == TREE_GATE_SIGMOID) return vfma(p, h - x, pick(p, h, x));
  return vfma(p, h, pick(p, h, vec<CH>(0.f)) + x);
}

DEVI float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
DEVI float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
DEVI float rcp_approx(float a) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(a));
  return r;
}
// e^n for -100 <= n <= 0: 2^t of the hardware (2 units in the last place) at t = n log2(e) rounded, and the
// first-order term of what the rounding took from n
template <int CH>
DEVI Vec<CH> exp_of(Vec<CH> n) {
  const Vec<CH> t = n * vec<CH>(1.4426950408889634f), r = vfma(t, vec<CH>(-0.6931471805599453f), n);
  Vec<CH> e;
#pragma unroll
  for (int c = 0; c < CH; ++c) e.v[c] = ex2_approx(t.v[c]);
  return vfma(e, r, e);
}
// p of gate values g
template <int KIND, int CH>
DEVI Vec<CH> gate_of(Vec<CH> g) {
  Vec<CH> n, p;
  if (KIND == TREE_GATE_SIGMOID) {
#pragma unroll
    for (int c = 0; c < CH; ++c) n.v[c] = max_nan(-fabsf(g.v[c]), -100.f);
    const Vec<CH> e = exp_of(n), d = e + vec<CH>(1.f);
    Vec<CH> q;
#pragma unroll
    for (int c = 0; c < CH; ++c) q.v[c] = rcp_approx(d.v[c]);
    q = e * q;                                        // the smaller of a and 1 - a; it is 1 - a where g >= 0
#pragma unroll
    for (int c = 0; c < CH; ++c)
      p.v[c] = __uint_as_float(__float_as_uint(q.v[c]) ^ (~__float_as_uint(g.v[c]) & 0x80000000u));
  } else {
#pragma unroll
    for (int c = 0; c < CH; ++c) n.v[c] = max_nan(min_nan(g.v[c], 0.f), -100.f);
    const Vec<CH> e = exp_of(n);
    // e^n - 1 for n > -ln 2: the series n + n^2/2! + ... + n^9/9!, whose next term is below 2^-26 of the sum
    Vec<CH> s = vec<CH>(1.f / 362880);
    s = vfma(s, n, vec<CH>(1.f / 40320));
    s = vfma(s, n, vec<CH>(1.f / 5040));
    s = vfma(s, n, vec<CH>(1.f / 720));
    s = vfma(s, n, vec<CH>(1.f / 120));
    s = vfma(s, n, vec<CH>(1.f / 24));
    s = vfma(s, n, vec<CH>(1.f / 6));
    s = vfma(s, n, vec<CH>(0.5f));
    s = vfma(n * n, s, n);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      p.v[c] = n.v[c] <= -0.6931471805599453f ? e.v[c] : __uint_as_float(__float_as_uint(s.v[c]) | 0x80000000u);
      if (g.v[c] > -0x1p-126f) p.v[c] = g.v[c] > 0.f ? __uint_as_float(kHeld) : -0.f;
    }
  }
  return p;
}

// A lane's word of a row: two bf16 channels or one fp32 channel.
template <typename T>
struct Lane;
template <>
struct Lane<__nv_bfloat16> {
  static constexpr int CH = 2;
  static DEVI Vec<2> unpack(uint32_t w) { return {{bf16lo(w), bf16hi(w)}}; }
  static DEVI uint32_t pack(Vec<2> a) { return pack_bf16(a.v[0], a.v[1]); }
};
template <>
struct Lane<float> {
  static constexpr int CH = 1;
  static DEVI Vec<1> unpack(uint32_t w) { return {{__uint_as_float(w)}}; }
  static DEVI uint32_t pack(Vec<1> a) { return __float_as_uint(a.v[0]); }
};
// fp32 values of a lane's channels, past L1 (another block may have written them)
// where `want`, else zeros; loads of a run of calls are all in flight before the first is used
DEVI Vec<2> ld_state_if(const float* p, bool want, Vec<2>) {
  Vec<2> r;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %3, 0;\n\tmov.f32 %0, 0f00000000;\n\tmov.f32 %1, 0f00000000;\n\t"
               "@q ld.global.cg.v2.f32 {%0, %1}, [%2];\n\t}"
               : "=&f"(r.v[0]), "=&f"(r.v[1]) : "l"(p), "r"((uint32_t)want) : "memory");
  return r;
}
DEVI Vec<1> ld_state_if(const float* p, bool want, Vec<1>) {
  Vec<1> r;
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\tmov.f32 %0, 0f00000000;\n\t"
               "@q ld.global.cg.f32 %0, [%1];\n\t}"
               : "=&f"(r.v[0]) : "l"(p), "r"((uint32_t)want) : "memory");
  return r;
}
DEVI void st_state(float* p, Vec<2> v) { __stcg(reinterpret_cast<float2*>(p), make_float2(v.v[0], v.v[1])); }
DEVI void st_state(float* p, Vec<1> v) { __stcg(p, v.v[0]); }
// Values that other blocks wait for: a lane's state, and its map h -> A h + B as (A, B) per channel.  Each
// word arrives by itself.
DEVI float full_word(float v) { return __float_as_uint(v) == kEmpty ? __uint_as_float(0x7fffffffu) : v; }
DEVI bool is_full(float v) { return __float_as_uint(v) != kEmpty; }
DEVI bool is_full(Vec<2> v) { return is_full(v.v[0]) && is_full(v.v[1]); }
DEVI bool is_full(Vec<1> v) { return is_full(v.v[0]); }
DEVI void hand_state(float* p, Vec<2> v) {
  asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(full_word(v.v[0])), "f"(full_word(v.v[1])) : "memory");
}
DEVI void hand_state(float* p, Vec<1> v) {
  asm volatile("st.relaxed.gpu.global.f32 [%0], %1;" ::"l"(p), "f"(full_word(v.v[0])) : "memory");
}
DEVI Vec<2> look_state(const float* p, Vec<2>) {
  Vec<2> r;
  asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(r.v[0]), "=f"(r.v[1]) : "l"(p) : "memory");
  return r;
}
DEVI Vec<1> look_state(const float* p, Vec<1>) {
  Vec<1> r;
  asm volatile("ld.relaxed.gpu.global.f32 %0, [%1];" : "=f"(r.v[0]) : "l"(p) : "memory");
  return r;
}
DEVI void hand_map(float* p, Vec<2> A, Vec<2> B) {
  asm volatile("st.relaxed.gpu.global.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(p), "f"(full_word(A.v[0])),
               "f"(full_word(B.v[0])), "f"(full_word(A.v[1])), "f"(full_word(B.v[1])) : "memory");
}
DEVI void hand_map(float* p, Vec<1> A, Vec<1> B) {
  asm volatile("st.relaxed.gpu.global.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(full_word(A.v[0])), "f"(full_word(B.v[0])) : "memory");
}
DEVI void look_map(const float* p, Vec<2>& A, Vec<2>& B) {
  asm volatile("ld.relaxed.gpu.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(A.v[0]), "=f"(B.v[0]), "=f"(A.v[1]), "=f"(B.v[1]) : "l"(p) : "memory");
}
DEVI void look_map(const float* p, Vec<1>& A, Vec<1>& B) {
  asm volatile("ld.relaxed.gpu.global.v2.f32 {%0, %1}, [%2];" : "=f"(A.v[0]), "=f"(B.v[0]) : "l"(p) : "memory");
}
template <int CH>
DEVI Vec<CH> sh_ld(const float* p) {
  Vec<CH> r;
  const int lane = threadIdx.x & 31;
  if constexpr (CH == 2) {
    const float2 a = reinterpret_cast<const float2*>(p)[lane];
    r.v[0] = a.x;
    r.v[1] = a.y;
  } else {
    r.v[0] = p[lane];
  }
  return r;
}
template <int CH>
DEVI void sh_st(float* p, Vec<CH> a) {
  const int lane = threadIdx.x & 31;
  if constexpr (CH == 2) reinterpret_cast<float2*>(p)[lane] = make_float2(a.v[0], a.v[1]);
  else p[lane] = a.v[0];
}

DEVI int ld_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
DEVI void set_release(int32_t* p, int bits) {      // *p |= bits, after everything before it
  asm volatile("red.release.gpu.global.or.b32 [%0], %1;" ::"l"(p), "r"(bits) : "memory");
}

// Wait for a phase of a barrier, the whole warp.  Most warps of a block wait most of the time, so a look at the
// barrier sleeps for up to kNap ns before it says no; the limit is looked at between naps.
constexpr uint32_t kNap = 20000;
DEVI bool wait_phase(uint64_t* bar, uint32_t parity, const WaitCtl& wc) {
  uint64_t t0 = 0;
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kNap)
        : "memory");
    if (__all_sync(0xffffffffu, ok)) return true;
    const uint64_t now = global_timer_ns();
    if (t0 == 0) t0 = now;
    const bool late = now - t0 > wc.limit_ns;
    if (__any_sync(0xffffffffu, late || *wc.abort_flag)) {
      if (late && wc.status) atomicExch(wc.status, TREE_ERR_TIMEOUT);
      *wc.abort_flag = 1;
      return false;
    }
  }
}

// Wait until look() is true.  The first wait of the grid that runs out of time stops all others.
template <typename Look>
DEVI bool wait_until(Look look, const WaitCtl& wc, int32_t* stop) {
  if (look()) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (look()) return true;
    if ((it & 15u) == 0) {
      if (*wc.abort_flag || ld_acquire(stop)) return false;
      if (global_timer_ns() - t0 > wc.limit_ns) {
        if (wc.status) atomicExch(wc.status, TREE_ERR_TIMEOUT);
        set_release(stop, 1);
        return false;
      }
    }
  }
}
// ... until a tile's node rows are written
DEVI bool wait_rows(const int32_t* flag, const WaitCtl& wc, int32_t* stop) {
  return wait_until([&] { return ld_acquire(flag) != 0; }, wc, stop);
}

DEVI void tma_load_2d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// A block works on up to SLOTS tiles at a time, in the order in which it drew them:
//   loading warp      draws a tile, starts its copies                                       -> full, told
//   mapping warps     the map of every token (backward: its p) and of every 16 tokens        -> mapped
//   publishing warp   joins the 16-token maps to the tile's, hands that to the other blocks  -> known
//   joining warp      finds the state before the tile, hands on the one behind it            -> ready
//   walking warps     wait for that state, write the results                                 -> empty
// So a tile whose state is late holds up nothing that another tile waits for: its map is out, and so are
// those of the tiles that the block drew after it.  Forward, 32768 tokens x 8192 channels bf16: 0.86 ms
// where one set of warps took a tile from its copies to its results, waiting in between.
template <int SLOTS>
struct ScanShared {
  uint64_t full[SLOTS], told[SLOTS], mapped[SLOTS], known[SLOTS], ready[SLOTS], empty[SLOTS];
  // Among the walking warps: done, a tile's rows are written (one for each slot: only one warp waits there, and
  // one that is a tile ahead must not be counted for this one); own, their own maps are there (all wait); turn,
  // the warp before is through.
  uint64_t done[SLOTS], own, turn[kScanWarps];
  int tile[SLOTS], slab[SLOTS], info[SLOTS], dist[SLOTS];
  int abort_flag;
  int reset[SLOTS][kScanWarps];
  alignas(16) float A[SLOTS][kScanWarps][64];      // per warp and channel: the map of its 16 tokens
  alignas(16) float B[SLOTS][kScanWarps][64];
  alignas(16) float all[SLOTS][2][64];             // the tile's map
  alignas(16) float in[SLOTS][64];                 // the state before (the gradient behind) the tile
  alignas(16) float carry[kScanWarps][64];         // the same for a warp, in tiles that go warp by warp
};
template <int SLOTS>
struct ScanBack {
  alignas(16) float R[SLOTS][kScanWarps][64];      // the gradient's map is u -> A u + R
  alignas(16) float before[kScanWarps][4][64];     // h before every fourth token, where it cannot stay in registers
};

// Forward: the states behind nodes that end in the tile at hand, one for every four tokens (the last that came).
struct ScanEnds {
  int token[TILE / 4];                             // which token's
  alignas(16) float state[TILE / 4][64];
};

constexpr int kSlots = 3, kPlanes = 4;             // 192 KB: a block an SM

template <typename T>
struct ScanFwd {
  const T *gate, *x;
  const float* init;
  T* y;
  float* states;
  ScanTree t;
  ScanWork w;
  int C, slabs;
  int32_t* status;
  uint64_t limit_ns;
};

template <typename T>
struct ScanBwd {
  const float *init, *states, *d_final;
  T *dgate, *dx;
  float* d_init;
  ScanTree t;
  ScanWork w;
  int C, slabs;
  int32_t* status;
  uint64_t limit_ns;
};

// The loading warp: draws tiles from the counter, starts their copies, and finds how many maps lie
// between the tile and the state it starts from.  FWD: that is the state behind the nearest tile before
// it that is no plain map or ends a group of kScanGroup; backward the same from the other side.
// Groups bound the maps that a tile joins; within one, no tile waits for a state to be handed on.
template <bool FWD, int TENSORS>
DEVI void scan_load(ScanShared<kSlots>& sh, uint8_t* slots, const CUtensorMap* const (&tm)[TENSORS], const ScanWork& w,
                    int tiles, int slabs, int slab_ch, bool joins, const WaitCtl& wc) {
  const int lane = threadIdx.x & 31;
  auto draw = [&] { return atomicAdd(reinterpret_cast<unsigned long long*>(w.ctl), 1ull); };
  unsigned long long next = lane == 0 ? draw() : 0;
  int i = 0, ends = 0;
  for (;; ++i) {
    const int s = i % kSlots;
    if (i >= kSlots && !wait_phase(&sh.empty[s], ((i / kSlots) - 1) & 1, wc)) break;
    const unsigned long long ticket = __shfl_sync(0xffffffffu, next, 0);
    const unsigned long long turn = ticket / (unsigned)slabs;    // tile by tile, its slabs side by side
    if (turn >= (unsigned)tiles) {                   // the end, for all that take tiles in turn
      if (lane == 0) {
        sh.tile[s] = -1;
        mbar_arrive(&sh.full[s]);
      }
      if (++ends == kEnds) break;
      continue;
    }
    const int slab = static_cast<int>(ticket - turn * (unsigned)slabs);
    const int k = FWD ? static_cast<int>(turn) : tiles - 1 - static_cast<int>(turn);
    if (lane == 0) {
      sh.tile[s] = k;
      sh.slab[s] = slab;
      mbar_expect_tx(&sh.full[s], TENSORS * kPlane);
#pragma unroll
      for (int a = 0; a < TENSORS; ++a)
        tma_load_2d(slots + (size_t)(s * kPlanes + a) * kPlane, tm[a], &sh.full[s], slab * slab_ch, k * TILE);
    }
    // The first tiles are drawn one at a time, so that neighbours go to different blocks; later ones ahead.
    if (i + 1 < kSlots && !wait_phase(&sh.full[s], 0, wc)) {
      ++i;
      break;
    }
    if (lane == 0) next = draw();
    const int j = FWD ? k - lane : k + lane;
    int info = (lane <= kScanGroup && j >= 0 && j < tiles) ? w.info[j] : kInfoBreak;
    // the mapping warps' maps hold: no break in the tile, and backward nothing that joins at a node's end
    const bool mapped = !(info & kInfoBreak) && (FWD || !(info & kInfoSource || (joins && (info & kInfoEnd))));
    const bool map = mapped && (FWD ? (j + 1) % kScanGroup != 0 : (info & kInfoOut) && j % kScanGroup != 0);
    const uint32_t run = __ballot_sync(0xffffffffu, map);
    if (lane == 0) {
      sh.info[s] = info | (mapped ? kInfoMapped : 0) | (map ? kInfoMap : 0);
      sh.dist[s] = __ffs(~(run >> 1)) - 1;
      mbar_arrive(&sh.told[s]);
    }
  }
  // every copy has landed before the block's shared memory goes, also where other warps gave up
  // (slots that hold an end had their copies used before)
  if (lane == 0)
    for (int q = max(0, i - kSlots); q < i; ++q) {
      const uint64_t t0 = global_timer_ns();
      while (sh.tile[q % kSlots] >= 0 && !mbar_try_wait(&sh.full[q % kSlots], (q / kSlots) & 1) &&
             global_timer_ns() - t0 < wc.limit_ns) {
      }
    }
}

// The next tile of a warp that is not the loading one; false at the end, or where a wait gave up.
struct Tile {
  int k, slab, info, dist, s;
  uint32_t parity;
};
DEVI bool next_tile(ScanShared<kSlots>& sh, int i, Tile& t, const WaitCtl& wc) {
  t.s = i % kSlots;
  t.parity = (i / kSlots) & 1;
  if (!wait_phase(&sh.full[t.s], t.parity, wc)) return false;
  t.k = sh.tile[t.s];
  t.slab = sh.slab[t.s];
  return t.k >= 0;
}
DEVI bool tile_info(ScanShared<kSlots>& sh, Tile& t, const WaitCtl& wc) {
  if (!wait_phase(&sh.told[t.s], t.parity, wc)) return false;
  t.info = sh.info[t.s];
  t.dist = sh.dist[t.s];
  return true;
}
DEVI void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A lane's words of a warp's 16 rows of a slot.  Planes 0, 1 (and backward 2) hold the tensors' rows.
// Forward, a token's map takes their place: A and B of the lane's first channel in planes 0 and 1, those of
// the second side by side in planes 2 and 3.  Backward, p does: first channel in plane 0, second in plane 3.
template <typename T>
struct Rows {
  uint8_t *base, *pair;
  static constexpr int CH = Lane<T>::CH;
  DEVI Rows(uint8_t* slots, int s, int warp) {
    const int lane = threadIdx.x & 31;
    base = slots + (size_t)s * kPlanes * kPlane + warp * kWarpTokens * kRow + lane * 4;
    pair = slots + ((size_t)s * kPlanes + 2) * kPlane + warp * kWarpTokens * 2 * kRow + lane * 8;
  }
  DEVI float& word(int plane, int i) const { return *reinterpret_cast<float*>(base + plane * kPlane + i * kRow); }
  DEVI Vec<CH> get(int plane, int i) const { return Lane<T>::unpack(__float_as_uint(word(plane, i))); }
  DEVI Vec<CH> p(int i) const {
    Vec<CH> r;
    r.v[0] = word(0, i);
    if constexpr (CH == 2) r.v[1] = word(3, i);
    return r;
  }
  DEVI void set_p(int i, Vec<CH> v) const {
    word(0, i) = v.v[0];
    if constexpr (CH == 2) word(3, i) = v.v[1];
  }
  DEVI void set_map(int i, Vec<CH> A, Vec<CH> B) const {
    word(0, i) = A.v[0];
    word(1, i) = B.v[0];
    if constexpr (CH == 2) *reinterpret_cast<float2*>(pair + i * 2 * kRow) = make_float2(A.v[1], B.v[1]);
  }
  DEVI Vec<CH> constant(int i) const {               // B alone
    Vec<CH> B;
    B.v[0] = word(1, i);
    if constexpr (CH == 2) B.v[1] = reinterpret_cast<const float2*>(pair + i * 2 * kRow)->y;
    return B;
  }
  DEVI Vec<CH> mapped(int i, Vec<CH> h) const {      // the token's map of the state before the warp
    Vec<CH> A, B;
    A.v[0] = word(0, i);
    B.v[0] = word(1, i);
    if constexpr (CH == 2) {
      const float2 m = *reinterpret_cast<const float2*>(pair + i * 2 * kRow);
      A.v[1] = m.x;
      B.v[1] = m.y;
    }
    return vfma(A, h, B);
  }
};

// The warp's writes so far, and those that a barrier ordered before them, become visible with the flag.
DEVI void publish(int32_t* flag) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) set_release(flag, 1);
}

// The state before a tile (backward: the gradient behind it), from the state behind tile b and the maps of the
// `dist` tiles between, in the order in which the recurrence passes them; b, b + step, ... lead to the tile.
// The maps are joined first, so that a state that arrives last is one step away from being handed on.
template <int CH>
struct Joiner {
  const ScanWork& w;
  int C, ch, b, step, dist;
  const float* state;                        // row of tile b, at the lane's channels
  bool on;
  DEVI const float* map(int j) const { return w.maps + ((size_t)(b + step * j) * C + ch) * 2; }
  // the joined state in v; false if a wait gave up
  DEVI bool join(Vec<CH>& v, const WaitCtl& wc) const {
    bool ok = true;
    if (on) {
      Vec<CH> A[kScanGroup - 1], B[kScanGroup - 1];
#pragma unroll
      for (int q = 1; q < kScanGroup; ++q)             // all loads first
        if (q <= dist) look_map(map(q), A[q - 1], B[q - 1]);
      v = look_state(state, v);
      Vec<CH> PA = vec<CH>(1.f), PB = vec<CH>(0.f);
#pragma unroll
      for (int q = 1; q < kScanGroup; ++q) {
        if (q > dist) break;
        if (ok && !(is_full(A[q - 1]) && is_full(B[q - 1])))
          ok = wait_until([&] { look_map(map(q), A[q - 1], B[q - 1]); return is_full(A[q - 1]) && is_full(B[q - 1]); },
                          wc, w.ctl + 2);
        PB = vfma(A[q - 1], PB, B[q - 1]);
        PA = PA * A[q - 1];
      }
      if (ok && !is_full(v)) ok = wait_until([&] { v = look_state(state, v); return is_full(v); }, wc, w.ctl + 2);
      if (dist) v = vfma(PA, v, PB);
    }
    return __all_sync(0xffffffffu, ok);
  }
};

// The publishing warp.  It waits for no other block, so that a tile's map is out as soon as it can be.
template <bool FWD, int CH>
DEVI void scan_publish(ScanShared<kSlots>& sh, const float (*add)[kScanWarps][64], const ScanWork& w, int C,
                       int slab_ch, const WaitCtl& wc) {
  const int lane = threadIdx.x & 31;
  Tile t;
  for (int i = 0; next_tile(sh, i, t, wc) && tile_info(sh, t, wc); ++i) {
    if (!wait_phase(&sh.mapped[t.s], t.parity, wc)) return;
    if (t.info & kInfoMapped) {
      Vec<CH> A = vec<CH>(1.f), B = vec<CH>(0.f);
#pragma unroll
      for (int n = 0; n < kScanWarps; ++n) {
        const int q = FWD ? n : kScanWarps - 1 - n;
        const Vec<CH> qa = sh_ld<CH>(sh.A[t.s][q]);
        B = vfma(qa, B, sh_ld<CH>(add[t.s][q]));
        A = A * qa;
      }
      const int ch = t.slab * slab_ch + lane * CH;
      if ((t.info & kInfoMap) && ch < C) hand_map(w.maps + ((size_t)t.k * C + ch) * 2, A, B);
      sh_st(sh.all[t.s][0], A);
      sh_st(sh.all[t.s][1], B);
    }
    warp_arrive(&sh.known[t.s]);
  }
}

// A joining warp.  rows: the states between tiles (backward: the gradients).
template <bool FWD, int CH>
DEVI void scan_join(ScanShared<kSlots>& sh, const ScanWork& w, int C, float* rows, int slab_ch, int joiner,
                    const WaitCtl& wc) {
  const int lane = threadIdx.x & 31;
  Tile t;
  for (int i = joiner; next_tile(sh, i, t, wc) && tile_info(sh, t, wc); i += kJoiners) {
    const int ch = t.slab * slab_ch + lane * CH;
    const bool on = ch < C, need = t.info & (FWD ? kInfoIn : kInfoOut);
    const int b = FWD ? t.k - 1 - t.dist : t.k + 1 + t.dist;
    const Joiner<CH> j{w, C, ch, b, FWD ? 1 : -1, t.dist, rows + (size_t)(need ? b : 0) * C + ch, on};
    Vec<CH> v = vec<CH>(0.f);
    if (need && !j.join(v, wc)) {
      if (lane == 0) sh.abort_flag = 1;
      return;
    }
    sh_st<CH>(sh.in[t.s], v);
    warp_arrive(&sh.ready[t.s]);
    if (!wait_phase(&sh.known[t.s], t.parity, wc)) return;
    if ((t.info & kInfoMapped) && on)
      hand_state(rows + (size_t)t.k * C + ch, vfma(sh_ld<CH>(sh.all[t.s][0]), v, sh_ld<CH>(sh.all[t.s][1])));
    warp_arrive(&sh.empty[t.s]);
  }
}

// The mapping warps, forward: every token's map of the state before its warp.
template <typename T, int KIND, int GROUPS>
DEVI void fwd_map(ScanShared<kSlots>& sh, uint8_t* slots, int group, int warp, const WaitCtl& wc) {
  constexpr int CH = Lane<T>::CH;
  Tile t;
  for (int i = group; next_tile(sh, i, t, wc); i += GROUPS) {
    const Rows<T> rows(slots, t.s, warp);
    Vec<CH> A = vec<CH>(1.f), B = vec<CH>(0.f);
#pragma unroll 4
    for (int q = 0; q < kWarpTokens; ++q) {
      const Vec<CH> p = gate_of<KIND>(rows.get(0, q));
      B = advance<KIND>(p, rows.get(1, q), B);
      A = decayed(p, A);
      rows.set_map(q, A, B);
    }
    sh_st(sh.A[t.s][warp], A);
    sh_st(sh.B[t.s][warp], B);
    fence_proxy_async_smem();                          // the maps lie where the next copies go
    warp_arrive(&sh.mapped[t.s]);
  }
}

// Forward, a warp whose 16 tokens hold breaks: the mapping warps' maps do not reach across one.  (Its loops are
// rolled: this is rare, and straight-line code for it would be fetched anew each time.)
template <typename T, int KIND>
struct FwdBreaks {
  static constexpr int CH = Lane<T>::CH;
  const ScanFwd<T>& a;
  const Rows<T>& rows;
  ScanEnds& kept;
  int k, t0, ch;
  bool on;
  int from, end;                           // per lane q < 16: link of token t0 + q, its node if it is the node's last
  uint32_t breaks, ends, reset;            // a bit a token; reset: breaks that start from outside the tile
  // New maps for the 16 tokens, from g and x in global memory, four at a time with their loads in flight
  // together.  Behind a break they start anew: from outside the tile with the state itself, as a constant in B;
  // from a node of this tile as maps of that node's state, which is not known yet.
  DEVI Vec<CH> remap(Vec<CH>& A) const {
    Vec<CH> B = vec<CH>(0.f);
    A = vec<CH>(1.f);
#pragma unroll 1
    for (int g = 0; g < kWarpTokens; g += 4) {
      Vec<CH> s[4];
      uint32_t gw[4], xw[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = __shfl_sync(0xffffffffu, from, g + q);
        const bool start = (reset >> (g + q)) & 1u;
        const float* row = n >= 0 ? a.states + (size_t)n * a.C
                                  : (a.init && start ? a.init + (size_t)a.t.tok_node[t0 + g + q] * a.C : nullptr);
        s[q] = ld_state_if(row + ch, on && row && start, B);
        const bool live = on && t0 + g + q < a.t.N;
        const size_t at = (size_t)(t0 + g + q) * a.C + ch;
        gw[q] = live ? *reinterpret_cast<const uint32_t*>(a.gate + at) : 0u;
        xw[q] = live ? *reinterpret_cast<const uint32_t*>(a.x + at) : 0u;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if ((breaks >> (g + q)) & 1u) {
          A = vec<CH>(1.f);
          B = ((reset >> (g + q)) & 1u) ? s[q] : vec<CH>(0.f);
        }
        const Vec<CH> p = gate_of<KIND>(Lane<T>::unpack(gw[q]));
        B = advance<KIND>(p, Lane<T>::unpack(xw[q]), B);
        A = decayed(p, A);
        rows.set_map(g + q, A, B);
      }
    }
    return B;
  }
  // The state that the run of tokens behind the break at q starts from, a node of this tile's.
  DEVI Vec<CH> source(int q) const {
    const int n = __shfl_sync(0xffffffffu, from, q);
    const int tok = a.t.tok_start[n] + a.t.node_len[n] - 1 - k * TILE, slot = tok / 4;
    if (kept.token[slot] == tok) return sh_ld<CH>(kept.state[slot]);
    return ld_state_if(a.states + (size_t)n * a.C + ch, on, Vec<CH>());     // another end has taken its place
  }
  DEVI void keep(int q, Vec<CH> v) const {   // the state of the node that ends at q
    const int e = __shfl_sync(0xffffffffu, end, q), tok = t0 + q - k * TILE, slot = tok / 4;
    if (on) st_state(a.states + (size_t)e * a.C + ch, v);
    sh_st(kept.state[slot], v);
    if ((threadIdx.x & 31) == 0) kept.token[slot] = tok;
    __syncwarp();
  }
  // Through the tokens at which something happens; h: the state before the warp.  Returns the state behind it.
  DEVI Vec<CH> pass(Vec<CH> h, bool keeping) const {
    bool set = false;                        // the run's states are in B already
    for (uint32_t m = (breaks & ~reset) | reset | (keeping ? ends : 0u); m; m &= m - 1) {
      const int q = __ffs(m) - 1;
      if ((breaks >> q) & 1u) {
        set = (reset >> q) & 1u;
        if (!set) h = source(q);
      }
      if ((ends >> q) & 1u) {
        const Vec<CH> v = set ? rows.constant(q) : rows.mapped(q, h);
        if (keeping) keep(q, v);
      }
    }
    return set ? rows.constant(kWarpTokens - 1) : rows.mapped(kWarpTokens - 1, h);
  }
  DEVI void write(Vec<CH> h) const {
    bool set = false;
#pragma unroll 1
    for (int q = 0; q < kWarpTokens; ++q) {
      if ((breaks >> q) & 1u) {
        set = (reset >> q) & 1u;
        if (!set) h = source(q);
      }
      const Vec<CH> v = set ? rows.constant(q) : rows.mapped(q, h);
      if (on && t0 + q < a.t.N) *reinterpret_cast<uint32_t*>(a.y + (size_t)(t0 + q) * a.C + ch) = Lane<T>::pack(v);
    }
  }
};

// The walking warps, forward.  Returns where a wait gave up or the tiles have ended.
template <typename T, int KIND>
DEVI void fwd_walk(const ScanFwd<T>& a, ScanShared<kSlots>& sh, ScanEnds& kept, uint8_t* slots, int warp,
                   const WaitCtl& wc) {
  constexpr int CH = Lane<T>::CH, SLAB = kRow / (int)sizeof(T);
  const int lane = threadIdx.x & 31;
  uint32_t n_own = 0, n_turn = 0;                      // uses of the walking warps' barriers so far
  Tile t;
  for (int i = 0; next_tile(sh, i, t, wc) && tile_info(sh, t, wc); ++i) {
    const Rows<T> rows(slots, t.s, warp);
    const int ch = t.slab * SLAB + lane * CH;          // the lane's first channel
    const int t0 = t.k * TILE + warp * kWarpTokens;
    FwdBreaks<T, KIND> f{a, rows, kept, t.k, t0, ch, ch < a.C, kLinkChain, -1, 0u, 0u, 0u};
    const bool serial = t.info & kInfoSerial;
    if (t.info & (kInfoBreak | kInfoEnd)) {
      bool ok = true, tile = false;
      if (lane < kWarpTokens && t0 + lane < a.t.N) {
        f.from = a.w.link[t0 + lane];
        f.end = a.w.end[t0 + lane];
        if (f.from >= 0) {
          const int ts = (a.t.tok_start[f.from] + a.t.node_len[f.from] - 1) / TILE;
          tile = ts == t.k;
          if (!tile) ok = wait_rows(a.w.flags + (size_t)ts * a.slabs + t.slab, wc, a.w.ctl + 2);
        }
      }
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) sh.abort_flag = 1;
        return;
      }
      f.breaks = __ballot_sync(0xffffffffu, f.from != kLinkChain);
      f.ends = __ballot_sync(0xffffffffu, f.end >= 0);
      f.reset = f.breaks & ~__ballot_sync(0xffffffffu, tile);
    }
    if (!wait_phase(&sh.mapped[t.s], t.parity, wc)) return;
    if (t.info & kInfoBreak) {
      if (f.breaks) {
        Vec<CH> A;
        const Vec<CH> B = f.remap(A);
        sh_st(sh.B[t.s][warp], B);                     // (a tile whose warps go one by one has no use for it)
      }
      if (lane == 0) sh.reset[t.s][warp] = f.breaks != 0;
      if (serial && lane < TILE / 4 / kScanWarps) kept.token[warp * (TILE / 4 / kScanWarps) + lane] = -1;
      // All maps are there; and no warp is a tile ahead, where its next turn would overtake this one's.
      warp_arrive(&sh.own);
      if (!wait_phase(&sh.own, n_own & 1, wc)) return;
      ++n_own;
    }
    // The state before the warp: from the maps of the warps before it; where a break starts from a node that
    // ends in this very tile, from the warp before it, which has then kept its nodes' states.
    Vec<CH> h;
    if (!serial) {
      Vec<CH> A = vec<CH>(1.f), B = vec<CH>(0.f);
      bool fixed = false;
#pragma unroll
      for (int q = 0; q < kScanWarps - 1; ++q) {
        if (q >= warp) break;
        const bool r = (t.info & kInfoBreak) && sh.reset[t.s][q];
        const Vec<CH> qa = sh_ld<CH>(sh.A[t.s][q]), qb = sh_ld<CH>(sh.B[t.s][q]);
        B = r ? qb : vfma(qa, B, qb);
        A = A * qa;
        fixed |= r;
      }
      if (!wait_phase(&sh.ready[t.s], t.parity, wc)) return;
      h = fixed ? B : vfma(A, sh_ld<CH>(sh.in[t.s]), B);
    } else {
      if (!wait_phase(&sh.ready[t.s], t.parity, wc)) return;
      if (warp > 0 && !wait_phase(&sh.turn[warp], n_turn & 1, wc)) return;
      ++n_turn;
      h = sh_ld<CH>(warp > 0 ? sh.carry[warp - 1] : sh.in[t.s]);
    }
    // first what others wait for: nodes' states, and the state behind the warp
    int32_t* flag = a.w.flags + (size_t)t.k * a.slabs + t.slab;
    if (t.info & (kInfoBreak | kInfoEnd)) {
      const Vec<CH> last = f.pass(h, true);
      if (serial && warp < kScanWarps - 1) {
        sh_st(sh.carry[warp], last);
        warp_arrive(&sh.turn[warp + 1]);
      }
      if ((t.info & kInfoBreak) && warp == kScanWarps - 1) {
        if (f.on) hand_state(a.states + (size_t)(a.t.n_nodes + t.k) * a.C + ch, last);
        if (serial) publish(flag);
      }
    }
    if (f.breaks) {
      f.write(h);
    } else {
      T* y = a.y + (size_t)t0 * a.C + ch;
      const int rest = f.on ? a.t.N - t0 : 0;          // tokens to write
#pragma unroll 4
      for (int q = 0; q < kWarpTokens; ++q, y += a.C) {
        const Vec<CH> v = rows.mapped(q, h);
        if (q < rest) *reinterpret_cast<uint32_t*>(y) = Lane<T>::pack(v);
      }
    }
    warp_arrive(&sh.done[t.s]);
    if (warp == 0 && !serial && (t.info & kInfoSource)) {      // breaks elsewhere start from nodes that end here
      if (!wait_phase(&sh.done[t.s], t.parity, wc)) return;
      publish(flag);
    }
    warp_arrive(&sh.empty[t.s]);
  }
}

// The mapping warps, backward: p, and the 16-token maps of h and of the gradient (which share the factor).
template <typename T, int KIND, int GROUPS>
DEVI void bwd_map(ScanShared<kSlots>& sh, ScanBack<kSlots>& back, uint8_t* slots, int group, int warp,
                  const WaitCtl& wc) {
  constexpr int CH = Lane<T>::CH;
  Tile t;
  for (int i = group; next_tile(sh, i, t, wc); i += GROUPS) {
    const Rows<T> rows(slots, t.s, warp);
    Vec<CH> A = vec<CH>(1.f), B = vec<CH>(0.f), R = vec<CH>(0.f);
#pragma unroll 4
    for (int q = 0; q < kWarpTokens; ++q) {
      const Vec<CH> p = gate_of<KIND>(rows.get(0, q));
      rows.set_p(q, p);
      B = advance<KIND>(p, rows.get(1, q), B);
      // the gradient's map, from the first token on: u before = R + A u behind
      R = vfma(decayed(p, A), rows.get(2, q), R);
      A = decayed(p, A);
    }
    sh_st(sh.A[t.s][warp], A);
    sh_st(sh.B[t.s][warp], B);
    sh_st(back.R[t.s][warp], R);
    fence_proxy_async_smem();
    warp_arrive(&sh.mapped[t.s]);
  }
}

// Backward, a warp at whose 16 tokens paths break or join.
template <typename T, int KIND>
struct BwdBreaks {
  static constexpr int CH = Lane<T>::CH;
  const ScanBwd<T>& a;
  const Rows<T>& rows;
  int t0, ch;
  bool on;
  int from, end, kid, sib, own;            // per lane q < 16, of token t0 + q; own: its node
  uint32_t breaks, joins;
  // h before four tokens from g on; h: before token g, and on return behind the four
  DEVI void befores(int g, Vec<CH>& h, Vec<CH> (&b)[4]) const {
    if ((breaks >> g) & 15u) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int n = __shfl_sync(0xffffffffu, from, g + q), v = __shfl_sync(0xffffffffu, own, g + q);
        const bool brk = (breaks >> (g + q)) & 1u;
        const float* row = n >= 0 ? a.states + (size_t)n * a.C : (a.init && brk ? a.init + (size_t)v * a.C : nullptr);
        b[q] = ld_state_if(row + ch, on && row && brk, h);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (!((breaks >> (g + q)) & 1u)) b[q] = h;
      h = advance<KIND>(rows.p(g + q), rows.get(1, g + q), b[q]);
    }
  }
  // dy of four tokens and what joins it: kid: the next node that starts from this one's state, with those behind
  // it; end: the node's own final state
  DEVI void sums(int g, Vec<CH> (&d)[4]) const {
#pragma unroll
    for (int q = 0; q < 4; ++q) d[q] = rows.get(2, g + q);
    if (!((joins >> g) & 15u)) return;
    Vec<CH> f[4], k[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int kd = __shfl_sync(0xffffffffu, kid, g + q), e = __shfl_sync(0xffffffffu, end, g + q);
      f[q] = ld_state_if(a.d_final + (size_t)e * a.C + ch, on && a.d_final && e >= 0, d[q]);
      k[q] = ld_state_if(a.w.dnode + (size_t)kd * a.C + ch, on && kd >= 0, d[q]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) d[q] = d[q] + (f[q] + k[q]);
  }
};

// The walking warps, backward: h before every token, then the gradients from the last token to the first.
template <typename T, int KIND>
DEVI void bwd_walk(const ScanBwd<T>& a, ScanShared<kSlots>& sh, ScanBack<kSlots>& back, uint8_t* slots, int warp,
                   const WaitCtl& wc) {
  constexpr int CH = Lane<T>::CH, SLAB = kRow / (int)sizeof(T);
  const int lane = threadIdx.x & 31;
  uint32_t n_own = 0, n_turn = 0;
  Tile t;
  for (int i = 0; next_tile(sh, i, t, wc) && tile_info(sh, t, wc); ++i) {
    const Rows<T> rows(slots, t.s, warp);
    const int ch = t.slab * SLAB + lane * CH;
    const int t0 = t.k * TILE + warp * kWarpTokens;
    int32_t* flag = a.w.flags + (size_t)t.k * a.slabs + t.slab;
    const bool mapped = t.info & kInfoMapped, serial = t.info & kInfoSerialBack;
    BwdBreaks<T, KIND> f{a, rows, t0, ch, ch < a.C, kLinkChain, -1, -1, -1, -1, 0u, 0u};
    const bool on = f.on;
    Vec<CH> h = ld_state_if(a.states + (size_t)(a.t.n_nodes + t.k - 1) * a.C + ch, on && (t.info & kInfoIn), Vec<CH>());
    if (!mapped) {
      bool ok = true;
      if (lane < kWarpTokens && t0 + lane < a.t.N) {
        const int j = t0 + lane;
        f.from = a.w.link[j];
        f.end = a.w.end[j];
        f.kid = a.w.kid[j];
        f.sib = a.w.sib[j];
        f.own = a.t.tok_node[j];
        if (f.kid >= 0) {
          const int tk = a.t.tok_start[f.kid] / TILE;
          if (tk != t.k) ok = wait_rows(a.w.flags + (size_t)tk * a.slabs + t.slab, wc, a.w.ctl + 2);
        }
        if (ok && f.sib >= 0) {
          const int tk = a.t.tok_start[f.sib] / TILE;
          if (tk != t.k) ok = wait_rows(a.w.flags + (size_t)tk * a.slabs + t.slab, wc, a.w.ctl + 2);
        }
      }
      if (!__all_sync(0xffffffffu, ok)) {
        if (lane == 0) sh.abort_flag = 1;
        return;
      }
      f.breaks = __ballot_sync(0xffffffffu, f.from != kLinkChain);
      f.joins = __ballot_sync(0xffffffffu, f.kid >= 0 || (f.end >= 0 && a.d_final));
    }
    const bool slow = f.breaks | f.joins;
    if (!wait_phase(&sh.mapped[t.s], t.parity, wc)) return;
    if (!mapped) {
      if (f.breaks) {                                  // h behind the warp does not depend on h before it
        Vec<CH> v = vec<CH>(0.f), b[4];
#pragma unroll 1
        for (int g = 0; g < kWarpTokens; g += 4) f.befores(g, v, b);
        sh_st(sh.B[t.s][warp], v);
      }
      if (slow && !serial) {
        Vec<CH> R = vec<CH>(0.f), d[4];
#pragma unroll 1
        for (int g = kWarpTokens - 4; g >= 0; g -= 4) {
          f.sums(g, d);
#pragma unroll
          for (int q = 3; q >= 0; --q) {
            R = decayed(rows.p(g + q), d[q] + R);
            if ((f.breaks >> (g + q)) & 1u) R = vec<CH>(0.f);
          }
        }
        sh_st(back.R[t.s][warp], R);
      }
      if (lane == 0) sh.reset[t.s][warp] = f.breaks != 0;
      warp_arrive(&sh.own);
      if (!wait_phase(&sh.own, n_own & 1, wc)) return;
      ++n_own;
    }
#pragma unroll
    for (int q = 0; q < kScanWarps - 1; ++q) {
      if (q >= warp) break;
      const Vec<CH> qb = sh_ld<CH>(sh.B[t.s][q]);
      h = (!mapped && sh.reset[t.s][q]) ? qb : vfma(sh_ld<CH>(sh.A[t.s][q]), h, qb);
    }
    // h before every fourth token; the others are stepped to again on the way back (16 values a lane would stay in
    // registers only in straight-line code of 15 KB, which the warps' other code would push out of the cache)
    if (!slow) {
#pragma unroll 4
      for (int q = 0; q < kWarpTokens - 4; ++q) {
        if (q % 4 == 0) sh_st(back.before[warp][q / 4], h);
        h = advance<KIND>(rows.p(q), rows.get(1, q), h);
      }
      sh_st(back.before[warp][3], h);
    } else {
      Vec<CH> b[4];
#pragma unroll 1
      for (int g = 0; g < kWarpTokens; g += 4) {
        sh_st(back.before[warp][g / 4], h);
        f.befores(g, h, b);
      }
    }
    // the gradient behind the warp, as the state before it in the forward
    Vec<CH> u;
    if (!serial) {
      Vec<CH> A = vec<CH>(1.f), R = vec<CH>(0.f);
      bool fixed = false;
#pragma unroll
      for (int q = kScanWarps - 1; q > 0; --q) {
        if (q <= warp) break;
        const bool r = !mapped && sh.reset[t.s][q];
        const Vec<CH> qa = sh_ld<CH>(sh.A[t.s][q]), qr = sh_ld<CH>(back.R[t.s][q]);
        R = r ? qr : vfma(qa, R, qr);
        A = A * qa;
        fixed |= r;
      }
      if (!wait_phase(&sh.ready[t.s], t.parity, wc)) return;
      u = fixed ? R : vfma(A, sh_ld<CH>(sh.in[t.s]), R);
    } else {
      if (!wait_phase(&sh.ready[t.s], t.parity, wc)) return;
      if (warp < kScanWarps - 1 && !wait_phase(&sh.turn[warp], n_turn & 1, wc)) return;
      ++n_turn;
      u = sh_ld<CH>(warp < kScanWarps - 1 ? sh.carry[warp + 1] : sh.in[t.s]);
    }
    // token q: lam = what reaches it; its gradients; u before it
    auto step = [&](int q, Vec<CH> lam, Vec<CH> before) {
      const Vec<CH> p = rows.p(q);
      u = decayed(p, lam);
      Vec<CH> dx, dg;
      if (KIND == TREE_GATE_SIGMOID) {
        Vec<CH> m;                                     // the smaller of a and 1 - a, and the larger
#pragma unroll
        for (int c = 0; c < CH; ++c) m.v[c] = fabsf(p.v[c]);
        const Vec<CH> l = vec<CH>(1.f) - m;
        dx = lam * pick(p, m, l);
        dg = lam * (m * l) * (before - rows.get(1, q));
      } else {
        dx = lam;
        dg = u * before;
#pragma unroll
        for (int c = 0; c < CH; ++c) dg.v[c] = __float_as_uint(p.v[c]) == kHeld ? 0.f : dg.v[c];
      }
      if (on && q < a.t.N - t0) {
        const size_t at = (size_t)(t0 + q) * a.C + ch;
        *reinterpret_cast<uint32_t*>(a.dgate + at) = Lane<T>::pack(dg);
        *reinterpret_cast<uint32_t*>(a.dx + at) = Lane<T>::pack(dx);
      }
    };
    if (!slow) {
#pragma unroll 1
      for (int g = kWarpTokens - 4; g >= 0; g -= 4) {
        Vec<CH> b[4];
        b[0] = sh_ld<CH>(back.before[warp][g / 4]);
#pragma unroll
        for (int q = 0; q < 3; ++q) b[q + 1] = advance<KIND>(rows.p(g + q), rows.get(1, g + q), b[q]);
#pragma unroll
        for (int q = 3; q >= 0; --q) step(g + q, rows.get(2, g + q) + u, b[q]);
      }
    } else {
#pragma unroll 1
      for (int g = kWarpTokens - 4; g >= 0; g -= 4) {
        Vec<CH> b[4], d[4], hg = sh_ld<CH>(back.before[warp][g / 4]);
        f.befores(g, hg, b);
        f.sums(g, d);
#pragma unroll
        for (int q = 3; q >= 0; --q) {
          const int kd = __shfl_sync(0xffffffffu, f.kid, g + q);
          // a node that starts within these four tokens hands its gradient on only now
          if (kd >= 0 && __any_sync(0xffffffffu, f.from != kLinkChain && f.own == kd && lane < kWarpTokens)) {
            const Vec<CH> again = ld_state_if(a.w.dnode + (size_t)kd * a.C + ch, on, u);
            const int e = __shfl_sync(0xffffffffu, f.end, g + q);
            const Vec<CH> own = ld_state_if(a.d_final + (size_t)e * a.C + ch, on && a.d_final && e >= 0, u);
            d[q] = rows.get(2, g + q) + (own + again);
          }
          step(g + q, d[q] + u, b[q]);
          if ((f.breaks >> (g + q)) & 1u) {            // what this path hands to the state it started from
            const int n = __shfl_sync(0xffffffffu, f.from, g + q), v = __shfl_sync(0xffffffffu, f.own, g + q);
            const int sb = __shfl_sync(0xffffffffu, f.sib, g + q);
            const Vec<CH> later = ld_state_if(a.w.dnode + (size_t)sb * a.C + ch, on && sb >= 0, u);
            if (on && n >= 0) st_state(a.w.dnode + (size_t)v * a.C + ch, u + later);
            if (on && n == kLinkRoot && a.d_init) st_state(a.d_init + (size_t)v * a.C + ch, u);
            u = vec<CH>(0.f);
          }
        }
      }
    }
    if (!mapped) {
      if (serial && warp > 0) {
        sh_st(sh.carry[warp], u);
        warp_arrive(&sh.turn[warp - 1]);
      }
      if (warp == 0) {
        if (on) hand_state(a.w.carry + (size_t)t.k * a.C + ch, u);
        if (serial) publish(flag);
      }
    }
    warp_arrive(&sh.done[t.s]);
    if (warp == 0 && !serial && (t.info & kInfoBreak)) {
      if (!wait_phase(&sh.done[t.s], t.parity, wc)) return;
      publish(flag);
    }
    warp_arrive(&sh.empty[t.s]);
  }
}

constexpr int kScanSmem = kSlots * kPlanes * kPlane + 1024;

DEVI uint8_t* scan_align(uint8_t* p) { return p + ((1024u - (smem_u32(p) & 1023u)) & 1023u); }

DEVI void scan_init(ScanShared<kSlots>& sh) {
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.told[s], 1);
      mbar_init(&sh.mapped[s], kScanWarps);
      mbar_init(&sh.known[s], 1);
      mbar_init(&sh.done[s], kScanWarps);
      mbar_init(&sh.ready[s], 1);
      mbar_init(&sh.empty[s], kScanWarps + 1);     // the walking warps and the joining warp
    }
    mbar_init(&sh.own, kScanWarps);
    for (int q = 0; q < kScanWarps; ++q) mbar_init(&sh.turn[q], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
}

// Every wait between warps is on an mbarrier and has a limit; the first that gives up raises the block's
// abort flag, which ends the others.
template <typename T, int KIND>
__global__ void __launch_bounds__(scan_threads(kFwdGroups), 1) k_scan_fwd(const __grid_constant__ CUtensorMap tm_gate,
                                                              const __grid_constant__ CUtensorMap tm_x,
                                                              const ScanFwd<T> a) {
  constexpr int CH = Lane<T>::CH, SLAB = kRow / (int)sizeof(T);
  extern __shared__ uint8_t smem_raw[];
  __shared__ ScanShared<kSlots> sh;
  __shared__ ScanEnds kept;
  uint8_t* slots = scan_align(smem_raw);
  scan_init(sh);
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  constexpr int WALK = kFwdGroups * kScanWarps, LOAD = WALK + kScanWarps;     // first warp of each role
  const int warp = threadIdx.x >> 5;
  if (warp < WALK) {
    fwd_map<T, KIND, kFwdGroups>(sh, slots, warp / kScanWarps, warp % kScanWarps, wc);
  } else if (warp < LOAD) {
    fwd_walk<T, KIND>(a, sh, kept, slots, warp - WALK, wc);
  } else if (warp == LOAD) {
    const CUtensorMap* tm[2] = {&tm_gate, &tm_x};
    scan_load<true>(sh, slots, tm, a.w, a.t.n_tiles, a.slabs, SLAB, false, wc);
  } else if (warp == LOAD + 1) {
    scan_publish<true, CH>(sh, sh.B, a.w, a.C, SLAB, wc);
  } else {
    scan_join<true, CH>(sh, a.w, a.C, a.states + (size_t)a.t.n_nodes * a.C, SLAB, warp - LOAD - 2, wc);
  }
}

template <typename T, int KIND>
__global__ void __launch_bounds__(scan_threads(kBwdGroups), 1) k_scan_bwd(const __grid_constant__ CUtensorMap tm_gate,
                                                              const __grid_constant__ CUtensorMap tm_x,
                                                              const __grid_constant__ CUtensorMap tm_dy,
                                                              const ScanBwd<T> a) {
  constexpr int CH = Lane<T>::CH, SLAB = kRow / (int)sizeof(T);
  extern __shared__ uint8_t smem_raw[];
  __shared__ ScanShared<kSlots> sh;
  __shared__ ScanBack<kSlots> back;
  uint8_t* slots = scan_align(smem_raw);
  scan_init(sh);
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  constexpr int WALK = kBwdGroups * kScanWarps, LOAD = WALK + kScanWarps;     // first warp of each role
  const int warp = threadIdx.x >> 5;
  if (warp < WALK) {
    bwd_map<T, KIND, kBwdGroups>(sh, back, slots, warp / kScanWarps, warp % kScanWarps, wc);
  } else if (warp < LOAD) {
    bwd_walk<T, KIND>(a, sh, back, slots, warp - WALK, wc);
  } else if (warp == LOAD) {
    const CUtensorMap* tm[3] = {&tm_gate, &tm_x, &tm_dy};
    scan_load<false>(sh, slots, tm, a.w, a.t.n_tiles, a.slabs, SLAB, a.d_final != nullptr, wc);
  } else if (warp == LOAD + 1) {
    scan_publish<false, CH>(sh, back.R, a.w, a.C, SLAB, wc);
  } else {
    scan_join<false, CH>(sh, a.w, a.C, a.w.carry, SLAB, warp - LOAD - 2, wc);
  }
}

// ---------------------------------------------------------------------------------------------
// host side

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// slabs of 128 bytes of channels: counted for the narrower type, which has the more of them
int scan_slabs(int C, int dtype) {
  const int per = kRow / (dtype == TREE_BF16 ? 2 : 4);
  return (C + per - 1) / per;
}

struct ScanLayout {
  size_t link, end, kid, sib, info, flags, ctl, maps, dnode, carry, total;
};

ScanLayout scan_layout(const tree_plan_t* p, int C) {
  ScanLayout L{};
  const size_t tok = align256((size_t)p->n_tokens * 4), tiles = (size_t)p->n_tiles;
  size_t o = 0;
  L.link = o;  o += tok;
  L.end = o;   o += tok;
  L.kid = o;   o += tok;
  L.sib = o;   o += tok;
  L.info = o;  o = align256(o + tiles * 4);
  L.flags = o; o = align256(o + tiles * scan_slabs(C, TREE_F32) * 4);
  L.ctl = o;   o = align256(o + 16);
  L.maps = o;  o = align256(o + tiles * C * 8);
  L.dnode = o; o = align256(o + (size_t)p->n_nodes * C * 4);
  L.carry = o; o = align256(o + tiles * C * 4);
  L.total = o;
  return L;
}

ScanWork scan_work(void* workspace, const ScanLayout& L) {
  uint8_t* w = static_cast<uint8_t*>(workspace);
  auto i32 = [&](size_t o) { return reinterpret_cast<int32_t*>(w + o); };
  auto f32 = [&](size_t o) { return reinterpret_cast<float*>(w + o); };
  return ScanWork{i32(L.link), i32(L.end), i32(L.kid), i32(L.sib), i32(L.info), i32(L.flags), i32(L.ctl),
                  f32(L.maps), f32(L.dnode), f32(L.carry)};
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

int scan_args(const tree_plan_t* plan, const int32_t* parent, const int32_t* node_len, int C, int dtype, int kind) {
  int rc = plan_ok(plan);
  if (rc) return rc;
  if (!plan->tok_node || !plan->tok_start || !plan->sub_end || !parent || !node_len) return TREE_ERR_ARG;
  if (plan->n_nodes <= 0 || C <= 0 || C % 8 != 0) return TREE_ERR_SHAPE;
  if ((dtype != TREE_BF16 && dtype != TREE_F32) || (kind != TREE_GATE_SIGMOID && kind != TREE_GATE_LOG))
    return TREE_ERR_SHAPE;
  return TREE_OK;
}

ScanTree scan_tree(const tree_plan_t* plan, const int32_t* parent, const int32_t* node_len) {
  return ScanTree{plan->tok_node, plan->tok_start, plan->sub_end, parent, node_len,
                  plan->n_tokens, plan->n_nodes,   plan->n_tiles};
}

// a tensor [N][C] in boxes of 128 tokens by a slab's channels; what lies outside reads as zero
template <typename T>
int scan_map(CUtensorMap* m, const void* base, int C, int N) {
  constexpr int box = kRow / (int)sizeof(T);
  return sizeof(T) == 2 ? make_tmap_bf16_2d(m, base, C, N, box, TILE) : make_tmap_f32_2d(m, base, C, N, box, TILE);
}

// A block an SM, or one for each unit of work.  The kernel's shared memory is announced once a device.
template <auto KERN>
int scan_grid(int64_t units, unsigned* blocks) {
  static std::atomic<int> sms_of[64];              // one array a kernel; 0: not announced yet
  int dev = 0, sms = 0;
  int rc = record_cuda(cudaGetDevice(&dev));
  if (rc) return rc;
  if (dev < 64) sms = sms_of[dev].load(std::memory_order_acquire);
  if (!sms) {
    rc = record_cuda(cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, kScanSmem));
    if (!rc) rc = record_cuda(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    if (rc) return rc;
    if (dev < 64) sms_of[dev].store(sms, std::memory_order_release);
  }
  *blocks = (unsigned)std::min<int64_t>(units, sms);
  return TREE_OK;
}

// 12 bytes a channel are marked empty for each tile: a block for 1024 channels
dim3 prepare_grid(const ScanTree& t, int C) { return dim3((unsigned)t.n_tiles, (unsigned)((C + 1023) / 1024)); }

template <typename T, int KIND>
int run_fwd(const ScanFwd<T>& a, const CUtensorMap& tg, const CUtensorMap& tx, cudaStream_t s) {
  unsigned blocks = 0;
  const int rc = scan_grid<&k_scan_fwd<T, KIND>>((int64_t)a.t.n_tiles * a.slabs, &blocks);
  if (rc) return rc;
  k_scan_fwd<T, KIND><<<blocks, scan_threads(kFwdGroups), kScanSmem, s>>>(tg, tx, a);
  return record_cuda(cudaGetLastError());
}
template <typename T, int KIND>
int run_bwd(const ScanBwd<T>& a, const CUtensorMap& tg, const CUtensorMap& tx, const CUtensorMap& td, cudaStream_t s) {
  unsigned blocks = 0;
  const int rc = scan_grid<&k_scan_bwd<T, KIND>>((int64_t)a.t.n_tiles * a.slabs, &blocks);
  if (rc) return rc;
  k_scan_bwd<T, KIND><<<blocks, scan_threads(kBwdGroups), kScanSmem, s>>>(tg, tx, td, a);
  return record_cuda(cudaGetLastError());
}

template <typename T>
int scan_fwd(const ScanTree& t, const ScanWork& w, const void* gate, const void* x, const float* init, int C, int dtype,
             int kind, void* y, float* states, int32_t* status, cudaStream_t s) {
  const int slabs = scan_slabs(C, dtype);
  CUtensorMap tg, tx;
  int rc = scan_map<T>(&tg, gate, C, t.N);
  if (!rc) rc = scan_map<T>(&tx, x, C, t.N);
  if (rc) return rc;
  k_scan_prepare<<<prepare_grid(t, C), TILE, 0, s>>>(t, w, slabs, C, 0, states, states + (size_t)t.n_nodes * C);
  const ScanFwd<T> a{static_cast<const T*>(gate), static_cast<const T*>(x), init, static_cast<T*>(y), states, t, w, C, slabs, status, wait_limit_ns()};
  return kind == TREE_GATE_SIGMOID ? run_fwd<T, TREE_GATE_SIGMOID>(a, tg, tx, s)
                                   : run_fwd<T, TREE_GATE_LOG>(a, tg, tx, s);
}

template <typename T>
int scan_bwd(const ScanTree& t, const ScanWork& w, const void* gate, const void* x, const float* init,
             const float* states, const void* dy, const float* d_final, int C, int dtype, int kind, void* dgate,
             void* dx, float* d_init, int32_t* status, cudaStream_t s) {
  const int slabs = scan_slabs(C, dtype);
  CUtensorMap tg, tx, td;
  int rc = scan_map<T>(&tg, gate, C, t.N);
  if (!rc) rc = scan_map<T>(&tx, x, C, t.N);
  if (!rc) rc = scan_map<T>(&td, dy, C, t.N);
  if (rc) return rc;
  k_scan_prepare<<<prepare_grid(t, C), TILE, 0, s>>>(t, w, slabs, C, 1, d_init, w.carry);
  const ScanBwd<T> a{init, states, d_final, static_cast<T*>(dgate), static_cast<T*>(dx), d_init, t, w, C, slabs, status,
                     wait_limit_ns()};
  return kind == TREE_GATE_SIGMOID ? run_bwd<T, TREE_GATE_SIGMOID>(a, tg, tx, td, s)
                                   : run_bwd<T, TREE_GATE_LOG>(a, tg, tx, td, s);
}

}  // namespace
}  // namespace ta

using namespace ta;

extern "C" {

size_t tree_scan_workspace(const tree_plan_t* plan, int C) {
  if (!plan || plan->n_tokens <= 0 || plan->n_nodes <= 0 || C <= 0) return 0;
  return scan_layout(plan, C).total;
}

int tree_scan_fwd(const tree_plan_t* plan, const int32_t* parent, const int32_t* node_len, const void* gate,
                  const void* x, const float* init, int C, int dtype, int gate_kind, void* workspace, void* y,
                  float* states, int32_t* status_dev, tree_stream_t stream) {
  int rc = scan_args(plan, parent, node_len, C, dtype, gate_kind);
  if (rc) return rc;
  for (const void* p : {gate, x, (const void*)workspace, (const void*)y, (const void*)states})
    if (!p || misaligned(p)) return TREE_ERR_ARG;
  if (init && misaligned(init)) return TREE_ERR_ARG;
  rc = check_device();
  if (rc) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const ScanTree t = scan_tree(plan, parent, node_len);
  const ScanWork w = scan_work(workspace, scan_layout(plan, C));
  return dtype == TREE_BF16
             ? scan_fwd<__nv_bfloat16>(t, w, gate, x, init, C, dtype, gate_kind, y, states, status_dev, s)
             : scan_fwd<float>(t, w, gate, x, init, C, dtype, gate_kind, y, states, status_dev, s);
}

int tree_scan_bwd(const tree_plan_t* plan, const int32_t* parent, const int32_t* node_len, const void* gate,
                  const void* x, const float* init, const float* states, const void* dy, const float* d_final, int C,
                  int dtype, int gate_kind, void* workspace, void* dgate, void* dx, float* d_init,
                  int32_t* status_dev, tree_stream_t stream) {
  int rc = scan_args(plan, parent, node_len, C, dtype, gate_kind);
  if (rc) return rc;
  for (const void* p : {gate, x, (const void*)states, dy, (const void*)workspace, (const void*)dgate, (const void*)dx})
    if (!p || misaligned(p)) return TREE_ERR_ARG;
  for (const void* p : {(const void*)init, (const void*)d_final, (const void*)d_init})
    if (p && misaligned(p)) return TREE_ERR_ARG;
  rc = check_device();
  if (rc) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const ScanTree t = scan_tree(plan, parent, node_len);
  const ScanWork w = scan_work(workspace, scan_layout(plan, C));
  return dtype == TREE_BF16
             ? scan_bwd<__nv_bfloat16>(t, w, gate, x, init, states, dy, d_final, C, dtype, gate_kind, dgate, dx, d_init,
                                       status_dev, s)
             : scan_bwd<float>(t, w, gate, x, init, states, dy, d_final, C, dtype, gate_kind, dgate, dx, d_init,
                               status_dev, s);
}

}  // extern "C"
