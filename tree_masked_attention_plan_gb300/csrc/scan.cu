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
// Measured (bf16, 268M elements, sigmoid gate): one sequence of 32768 tokens by 8192 channels forward
// 0.34 ms, 4.8 TB/s, backward 0.57 ms, 4.7 TB/s; a tree of the same size (nodes of some 250 tokens) 0.39 and
// 0.70 ms.  What bounds it there is instruction issue and the dependent steps of a warp's walk (in the backward a
// step of 64 channels takes 109 instructions, and the SM issues in 62 % of all cycles; the copies alone, without
// the arithmetic, take 0.27 ms in the forward).  In a tree of short nodes it is the way of a state through tiles in
// which a break starts from a node that ends there too: they hand on a state, warp by warp, 3.5 us a tile (a tile
// without breaks hands on its map: 0.4).  3456 tokens of a caterpillar by 4096 channels take 95 us, 13 at the
// memory's rate.
// Why 128 tokens: a tile hands on 4 bytes of state and 8 of map for each channel, and one of 64 tokens twice as
// often (the tree: 0.53 instead of 0.42 ms forward, 1.00 instead of 0.78 backward).
//
// Precision: states, gates and gradients are fp32.  The forward holds a and the input's weight apart, each to the
// accuracy that token_of states.  The backward has one word for both: p = -(1 - a) where a > 1/2, p = a elsewhere, so
// that neither the little that a long memory loses a token nor a small decay drowns in the other's rounding; it computes
// h again with that, from the forward's state before the tile, so that within a tile the two differ by roundings of a.
#include <algorithm>
#include <atomic>

#include "common.cuh"

namespace ta {
int make_tmap_bf16_2d(CUtensorMap* m, const void* base, int inner, int rows, int box_inner, int box_rows);  // host.cu

namespace {

constexpr int kTile = TREE_SCAN_TILE;       // tokens of a tile
constexpr int kScanWarps = 8;               // warps that share a tile: 16 tokens each
constexpr int kSlots = 3, kPlanes = 4;       // tiles that a block holds, 64 KB each: a block an SM
// A block: eight mapping warps, eight walking warps, one warp that loads, one that publishes, two that join, which take
// tiles in turn (three cost the backward a tenth).  Sixteen mapping warps in the forward: one sequence of 32768 x 8192
// in 0.33 ms instead of 0.34, but trees (which the walking warps bound) slower, the caterpillar 115 us instead of 103.
// A second group of walking warps in the backward leaves 72 registers a thread, which spill: the rollout 0.95 -> 1.72 ms.
constexpr int kJoins = 2, kScanThreads = 32 * (2 * kScanWarps + 2 + kJoins);
constexpr int kWarpTokens = kTile / kScanWarps;
constexpr int kRow = 128;                   // bytes of a tile's row: 64 bf16 or 32 fp32 channels, a word a lane
constexpr int kPlane = kTile * kRow;         // one tensor's rows of a tile
constexpr int kScanGroup = 4;               // at most this many maps are joined to a state (8: 131072 x 2048 2 % slower)

constexpr int kMostChannels = 1 << 28;      // a row's bytes and the channels behind its last slab still count as int

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
// info, edge: per tile, the kInfo bits; its first and last break (bits 0-7, 8-15).  ctl: the counter that hands out tiles (64 bits), and a word that stops every
// wait once one has run out of time.  dnode: per node that starts at a break, the gradient that it and the nodes
// behind it hand to the state they start from.
struct ScanWork {
  int32_t *link, *end, *kid, *sib, *info, *edge, *ctl;
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
  kInfoLast = 512,      // its last break starts from outside the tile
  kInfoFirst = 1024,    // nothing joins before its first break but nodes' final states
  kInfoFirstEnd = 2048, // a node ends before its first break
};
// What tiles hand to one another carries its own arrival: the rows of maps, of the states between tiles, of nodes
// that breaks start from (backward: dnode) hold this pattern, a NaN that no arithmetic gives, until they are written,
// and whoever needs one polls the value itself.  No flag and no fence stands between a tile and the next: with
// flags for the nodes' rows the 20011 x 1000 forest took 0.90 ms a step instead of 0.73.
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

// a node that a break starts from: its first child follows on it, a further one starts behind that
DEVI bool is_source(int v, const ScanTree& t) {
  const int next = t.tok_start[v] + t.node_len[v];
  return next < t.sub_end[v] && t.sub_end[t.tok_node[next]] < t.sub_end[v];
}

// Blocks (tile, 0): links and info.  Blocks (tile, share of the channels from 1 on): the tile's map and the state behind it marked empty.  FWD:
// states of nodes that breaks start from marked empty, of nodes without tokens zeroed.  Backward: dnode of nodes
// that start at a break from another's state marked empty, d_init of those that do not start from it zeroed.
template <bool FWD>
__global__ void __launch_bounds__(kTile) k_scan_prepare(ScanTree t, ScanWork w, int C, float* rows, float* between) {
  __shared__ int bits, lo, hi;
  __shared__ uint8_t marks[kTile];
  const int k = blockIdx.x, j = k * kTile + threadIdx.x;
  if (blockIdx.y) {
    const uint4 e = make_uint4(kEmpty, kEmpty, kEmpty, kEmpty);
    const int first = (blockIdx.y - 1) * kTile + threadIdx.x, step = (gridDim.y - 1) * kTile;
    uint4* m = reinterpret_cast<uint4*>(w.maps + (size_t)k * C * 2);
    uint4* b = reinterpret_cast<uint4*>(between + (size_t)k * C);
    for (int i = first; i < C / 2; i += step) m[i] = e;
    for (int i = first; i < C / 4; i += step) b[i] = e;
    auto fill = [&](float* row, uint4 v) {
      for (int i = first; i < C / 4; i += step) reinterpret_cast<uint4*>(row)[i] = v;
    };
    // a node a thread, then a row at a time
    enum : uint8_t { kNone = 0, kRowEmpty = 1, kRowZero = 2 };
    for (int v0 = k * kTile; v0 < t.n_nodes; v0 += gridDim.x * kTile) {
      const int v = v0 + threadIdx.x;
      uint8_t mark = kNone;
      if (v < t.n_nodes) {
        const bool some = t.node_len[v] > 0;
        if (FWD) {
          mark = !some ? kRowZero : is_source(v, t) ? kRowEmpty : kNone;
        } else {
          const int link = some ? link_of(t.tok_start[v], t) : kLinkChain;
          mark = (link >= 0 ? kRowEmpty : kNone) | (rows && link != kLinkRoot ? kRowZero : kNone);
        }
      }
      marks[threadIdx.x] = mark;
      __syncthreads();
      for (int q = 0; q < min(kTile, t.n_nodes - v0); ++q) {
        const size_t at = (size_t)(v0 + q) * C;
        if (marks[q] & kRowEmpty) fill((FWD ? rows : w.dnode) + at, e);
        if (marks[q] & kRowZero) fill(rows + at, make_uint4(0, 0, 0, 0));
      }
      __syncthreads();
    }
    return;
  }
  if (threadIdx.x == 0) {
    bits = 0;
    lo = kTile;
    hi = -1;
  }
  if (k == 0 && threadIdx.x < 4) w.ctl[threadIdx.x] = 0;
  __syncthreads();
  int mine = 0, kid = -1, end = -1;
  bool outside = true;
  if (j < t.N) {
    const int v = t.tok_node[j];
    const int link = link_of(j, t);
    int sib = -1;
    if (link != kLinkChain) {
      mine |= kInfoBreak;
      atomicMin(&lo, (int)threadIdx.x);
      atomicMax(&hi, (int)threadIdx.x);
    } else if (threadIdx.x == 0) mine |= kInfoIn;
    if (link >= 0) {
      if ((t.tok_start[link] + t.node_len[link] - 1) / kTile == k) {
        mine |= kInfoSerial;
        outside = false;
      }
      const int next = t.sub_end[v];
      if (next < t.sub_end[link]) {
        sib = t.tok_node[next];
        if (next / kTile == k) mine |= kInfoSerialBack;
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
          if (next / kTile == k) mine |= kInfoSerialBack;
        }
      }
    }
    if (threadIdx.x == kTile - 1 && j + 1 < t.N && link_of(j + 1, t) == kLinkChain) mine |= kInfoOut;
    w.link[j] = link;
    w.end[j] = end;
    w.kid[j] = kid;
    w.sib[j] = sib;
  }
  __syncthreads();
  if ((int)threadIdx.x == hi && outside) mine |= kInfoLast;
  if ((int)threadIdx.x < lo && end >= 0) mine |= kInfoFirstEnd;
  if (mine) atomicOr(&bits, mine);
  const bool kids = __syncthreads_or((int)threadIdx.x < lo && kid >= 0);
  if (threadIdx.x == 0) {
    w.info[k] = bits | (hi >= 0 && !kids ? kInfoFirst : 0);
    w.edge[k] = (lo & 255) | (max(hi, 0) << 8);
  }
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
// e^n for -100 <= n <= 87: 2^t of the hardware (2 units in the last place) at t = n log2(e) rounded, and the
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

// The forward's form of a token: decay a and input b.  Sigmoid: a = 1 / (1 + e) and 1 - a = e / (1 + e) with
// e = e^-g; g is held above -87, where e is still finite and a already below 2e-38.
// fp32 tensors (EXACT): e as exp_of has it, so that a and 1 - a are right to 13 units of 2^-24 of their own size.  bf16
// tensors: what the rounding of -g log2(e) takes is left out, 1 unit for each unit of |g| or so (17 at 16, 62 at 87): the
// gate itself came with some 2^15 times as much.  With it one sequence of 32768 x 8192 takes 352 us instead of 338, the rollout
// 398 instead of 388.
// Log: b = x and a = 1 + p.  a is fp32 as the state is, so that a token may cost a state 2^-25 twice over, once in a and
// once in a h + b: at memories of 2^20 tokens the rate is off by a thirtieth, and 1 - a below 2^-25 is lost.  p in its
// place would not help: the product of decays that a map is made of is rounded in the same way.
template <int KIND, bool EXACT, int CH>
DEVI void token_of(Vec<CH> g, Vec<CH> x, Vec<CH>& a, Vec<CH>& b) {
  if (KIND == TREE_GATE_SIGMOID) {
    Vec<CH> n, e;
    if (EXACT) {
#pragma unroll
      for (int c = 0; c < CH; ++c) n.v[c] = min_nan(max_nan(-g.v[c], -100.f), 87.f);
      e = exp_of(n);
    } else {
#pragma unroll
      for (int c = 0; c < CH; ++c) n.v[c] = max_nan(g.v[c], -87.f);
      n = n * vec<CH>(-1.4426950408889634f);
#pragma unroll
      for (int c = 0; c < CH; ++c) e.v[c] = ex2_approx(n.v[c]);
    }
    const Vec<CH> d = e + vec<CH>(1.f);
#pragma unroll
    for (int c = 0; c < CH; ++c) a.v[c] = rcp_approx(d.v[c]);
    b = (e * a) * x;
  } else {
    const Vec<CH> p = gate_of<TREE_GATE_LOG>(g);
    a = p + pick(p, vec<CH>(1.f), vec<CH>(0.f));
    b = x;
  }
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
// the same through L1, of what no block of the kernel writes
DEVI Vec<2> ld_given_if(const float* p, bool want, Vec<2>) {
  const float2 a = want ? __ldg(reinterpret_cast<const float2*>(p)) : make_float2(0.f, 0.f);
  return {{a.x, a.y}};
}
DEVI Vec<1> ld_given_if(const float* p, bool want, Vec<1>) { return {{want ? __ldg(p) : 0.f}}; }
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
constexpr uint64_t kDrainNs = 2000000000;           // for a block's copies in flight (they land within microseconds)
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
DEVI void tma_load_2d(void* dst, const CUtensorMap* m, uint64_t* bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(smem_u32(bar))
      : "memory");
}

// A block works on up to kSlots tiles at a time, in the order in which it drew them:
//   loading warp      draws a tile, starts its copies, looks up what it holds               -> full, told
//   mapping warps     the map of every token (backward: its p) and of every warp's tokens    -> mapped
//   publishing warp   joins the warps' maps to the tile's, hands that to the other blocks
//                     (`cut`: or at once what the tile hands on)                             -> known
//   joining warp      finds the state before the tile, hands on the one behind it            -> ready
//   walking warps     wait for that state, write the results                                 -> empty
// So a tile whose state is late holds up nothing that another tile waits for: its map is out, and so are
// those of the tiles that the block drew after it.
struct ScanShared {
  uint64_t full[kSlots], told[kSlots], mapped[kSlots], known[kSlots], ready[kSlots], empty[kSlots];
  int tile[kSlots], slab[kSlots], info[kSlots];
  int dist[kSlots];                                // maps between the tile and the state that it starts from
  int cut[kSlots];                                 // the break that decides what the tile hands on, -1: see scan_load
  int handed[kSlots];                              // the publishing warp has handed it on
  int abort_flag;
  int reset[kSlots][kScanWarps];
  // Per warp and channel the map of its tokens; in a tile without breaks the publishing warp puts that of all
  // tokens before the warp there (backward: in B the state before it, in A and R the gradient's map behind it).
  alignas(16) float A[kSlots][kScanWarps][64];
  alignas(16) float B[kSlots][kScanWarps][64];
  alignas(16) float all[kSlots][2][64];             // the tile's map
  alignas(16) float in[kSlots][64];                 // the state before (the gradient behind) the tile
};
// The walking warps among themselves.
struct ScanWalk {
  uint64_t own, turn[kScanWarps];                  // all of them are here; carry of the warp before is there
  alignas(16) float carry[kScanWarps][64];         // the state before (gradient behind) a warp, where they go one by one
  // The last such tile (counted from 1) in which token i's row (forward: the state of the node that ends there,
  // backward: the gradient that the node that starts there hands on) was written: warps of one tile wait for it.
  int row_of[kTile];
};
struct ScanBack {
  alignas(16) float R[kSlots][kScanWarps][64];      // the gradient's map is u -> A u + R
  alignas(16) float before[kScanWarps][kWarpTokens / 4][64];     // h before every fourth token, where it cannot stay in registers
};

// the warp's row of token tok (and what it wrote before) is there for the other warps of the block
DEVI void row_written(ScanWalk& walk, int tok, int serial) {
  __threadfence_block();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) *(volatile int*)&walk.row_of[tok] = serial;
}

// Forward: the states behind nodes that end in the tile at hand, one for every kKeep tokens (the last that came).
constexpr int kKeep = 8;
struct ScanEnds {
  int token[kTile / kKeep];                         // which token's
  alignas(16) float state[kTile / kKeep][64];
};

template <typename T>
struct ScanFwd {
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

// The loading warp: draws tiles from the counter and starts their copies.
template <bool FWD, int TENSORS>
DEVI void scan_load(ScanShared& sh, uint8_t* slots, const CUtensorMap* const (&tm)[TENSORS], const ScanWork& w,
                    int tiles, int slabs, int slab_ch, bool joins, const WaitCtl& wc) {
  const int lane = threadIdx.x & 31;
  unsigned long long turn = 0;
  int slab = 0, k = 0, mine = 0, edge = 0;
  // draws the next tile and looks up what it and its neighbours hold, ahead of the slot that it will take
  auto draw = [&] {
    unsigned long long ticket = 0;
    if (lane == 0) ticket = atomicAdd(reinterpret_cast<unsigned long long*>(w.ctl), 1ull);
    ticket = __shfl_sync(0xffffffffu, ticket, 0);
    // tile by tile, its slabs side by side
    turn = ticket >> 32 ? ticket / (unsigned)slabs : (uint32_t)ticket / (uint32_t)slabs;
    if (turn >= (unsigned)tiles) return;
    slab = static_cast<int>(ticket - turn * (unsigned)slabs);
    k = FWD ? static_cast<int>(turn) : tiles - 1 - static_cast<int>(turn);
    const int n = FWD ? k - lane : k + lane;
    mine = (lane <= kScanGroup && n >= 0 && n < tiles) ? w.info[n] : kInfoBreak;
    edge = w.edge[k];
  };
  draw();
  int i = 0, ends = 0;
  for (;; ++i) {
    const int s = i % kSlots;
    if (i >= kSlots && !wait_phase(&sh.empty[s], ((i / kSlots) - 1) & 1, wc)) break;
    if (turn >= (unsigned)tiles) {                   // the end, for all that take tiles in turn
      if (lane == 0) {
        sh.tile[s] = -1;
        mbar_arrive(&sh.told[s]);
        mbar_arrive(&sh.full[s]);
      }
      if (++ends == kSlots) break;
      continue;
    }
    const int n = FWD ? k - lane : k + lane;
    int info = mine;
    // the mapping warps' maps hold: no break in the tile, and backward nothing that joins at a node's end
    const bool mapped = !(info & kInfoBreak) && (FWD || !(info & kInfoSource || (joins && (info & kInfoEnd))));
    const bool map = mapped && (FWD ? (n + 1) % kScanGroup != 0 : (info & kInfoOut) && n % kScanGroup != 0);
    const uint32_t run = __ballot_sync(0xffffffffu, map);
    info = __shfl_sync(0xffffffffu, info | (mapped ? kInfoMapped : 0) | (map ? kInfoMap : 0), 0);
    // The tile's last break (backward: the first) where what the tile hands on is a plain map of what that break
    // starts from (is known from the tokens before it): it is handed on before the tile is walked, whose turn comes
    // after those of the block's earlier tiles (32768 x 2048 rollout: 210 -> 142 us forward, 342 -> 326 backward).
    const bool cut = FWD ? info & kInfoLast : (info & kInfoFirst) && !(joins && (info & kInfoFirstEnd));
    if (lane == 0) {                                 // (all of it there for those who wait for `full`, too)
      sh.tile[s] = k;
      sh.slab[s] = slab;
      sh.info[s] = info;
      sh.cut[s] = !cut ? -1 : FWD ? edge >> 8 : edge & 255;
      sh.dist[s] = __ffs(~(run >> 1)) - 1;
      mbar_arrive(&sh.told[s]);
      mbar_expect_tx(&sh.full[s], TENSORS * kPlane);
#pragma unroll
      for (int a = 0; a < TENSORS; ++a)
        tma_load_2d(slots + (size_t)(s * kPlanes + a) * kPlane, tm[a], &sh.full[s], slab * slab_ch, k * kTile);
    }
    // The first tiles are drawn one at a time, so that neighbours go to different blocks; later ones ahead.
    if (i + 1 < kSlots && !wait_phase(&sh.full[s], 0, wc)) {
      ++i;
      break;
    }
    draw();
  }
  // every copy has landed before the block's shared memory goes, also where other warps gave up
  // (slots that hold an end had their copies used before); the limit that a caller sets for waits does not shorten this one
  if (lane == 0)
    for (int q = max(0, i - kSlots); q < i; ++q) {
      const uint64_t t0 = global_timer_ns();
      while (sh.tile[q % kSlots] >= 0 && !mbar_try_wait(&sh.full[q % kSlots], (q / kSlots) & 1) &&
             global_timer_ns() - t0 < max(wc.limit_ns, kDrainNs)) {
      }
    }
}

// The next tile of a warp that is not the loading one; false at the end, or where a wait gave up.
struct Tile {
  int k, slab, info, s;
  uint32_t parity;
};
// `bar`: what of the tile is waited for; a tile number of -1 there is the end
DEVI bool next_tile(const ScanShared& sh, uint64_t (&bar)[kSlots], int i, Tile& t, const WaitCtl& wc) {
  t.s = i % kSlots;
  t.parity = (i / kSlots) & 1;
  if (!wait_phase(&bar[t.s], t.parity, wc)) return false;
  t.k = sh.tile[t.s];
  t.slab = sh.slab[t.s];
  t.info = sh.info[t.s];
  return t.k >= 0;
}
DEVI void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A lane's words of a warp's 16 rows of a slot.  Planes 0, 1 (and backward 2) hold the tensors' rows.  Forward,
// a and b take their place: those of the lane's first channel in planes 0 and 1, of the second side by side in
// planes 2 and 3.  Backward, p does: first channel in plane 0, second in plane 3.
template <typename T>
struct Rows {
  uint8_t *base, *pair;
  static constexpr int CH = Lane<T>::CH;
  DEVI Rows(uint8_t* slots, int s, int warp) {
    const int lane = threadIdx.x & 31, row = warp * kWarpTokens;
    base = slots + (size_t)s * kPlanes * kPlane + row * kRow + lane * 4;
    pair = slots + ((size_t)s * kPlanes + 2) * kPlane + row * 2 * kRow + lane * 8;
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
  DEVI void set_token(int i, Vec<CH> a, Vec<CH> b) const {
    word(0, i) = a.v[0];
    word(1, i) = b.v[0];
    if constexpr (CH == 2) *reinterpret_cast<float2*>(pair + i * 2 * kRow) = make_float2(a.v[1], b.v[1]);
  }
  DEVI Vec<CH> decay(int i) const {
    Vec<CH> a;
    a.v[0] = word(0, i);
    if constexpr (CH == 2) a.v[1] = *reinterpret_cast<const float*>(pair + i * 2 * kRow);
    return a;
  }
  DEVI Vec<CH> step(int i, Vec<CH> h) const {        // a h + b
    Vec<CH> a, b;
    a.v[0] = word(0, i);
    b.v[0] = word(1, i);
    if constexpr (CH == 2) {
      const float2 m = *reinterpret_cast<const float2*>(pair + i * 2 * kRow);
      a.v[1] = m.x;
      b.v[1] = m.y;
    }
    return vfma(a, h, b);
  }
};

// a row that another tile may still have to write: wait until it is there, after a first look at it in v
template <int CH>
DEVI bool arrived(const float* row, Vec<CH>& v, bool want, const WaitCtl& wc, int32_t* stop) {
  if (!want || is_full(v)) return true;
  return wait_until([&] { v = look_state(row, v); return is_full(v); }, wc, stop);
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

// The state that the break at token j starts from, in v.  Not null: where it is polled (it is another tile's to write)
template <typename T, int CH>
DEVI const float* cut_row(const ScanFwd<T>& a, int j, int ch, Vec<CH>& v) {
  const int n = a.w.link[j];
  const bool on = ch < a.C;
  const float* row = a.states + (size_t)max(n, 0) * a.C + ch;
  v = vec<CH>(0.f);
  if (n >= 0 && on) v = look_state(row, v);
  if (n < 0 && a.init) v = ld_state_if(a.init + (size_t)a.t.tok_node[j] * a.C + ch, on, v);
  return n >= 0 && on ? row : nullptr;
}

// The publishing warp.  It waits for no other block, so that a tile's map is out as soon as it can be.
template <typename T>
DEVI void fwd_publish(const ScanFwd<T>& a, ScanShared& sh, int slab_ch, const WaitCtl& wc) {
  constexpr int CH = Lane<T>::CH;
  const ScanWork& w = a.w;
  const int lane = threadIdx.x & 31, C = a.C;
  Tile t;
  for (int i = 0; next_tile(sh, sh.told, i, t, wc); ++i) {
    if (!wait_phase(&sh.mapped[t.s], t.parity, wc)) return;
    const int ch = t.slab * slab_ch + lane * CH, cut = sh.cut[t.s];
    if (t.info & kInfoMapped) {
      Vec<CH> A = vec<CH>(1.f), B = vec<CH>(0.f);
#pragma unroll 8
      for (int q = 0; q < kScanWarps; ++q) {
        const Vec<CH> qa = sh_ld<CH>(sh.A[t.s][q]), qb = sh_ld<CH>(sh.B[t.s][q]);
        sh_st(sh.A[t.s][q], A);
        sh_st(sh.B[t.s][q], B);
        B = vfma(qa, B, qb);
        A = A * qa;
      }
      if ((t.info & kInfoMap) && ch < C) hand_map(w.maps + ((size_t)t.k * C + ch) * 2, A, B);
      sh_st(sh.all[t.s][0], A);
      sh_st(sh.all[t.s][1], B);
    } else if (cut >= 0) {
      Vec<CH> A = vec<CH>(1.f), B = vec<CH>(0.f);
      for (int q = cut / kWarpTokens; q < kScanWarps; ++q) {
        const Vec<CH> qa = sh_ld<CH>(sh.A[t.s][q]);
        B = vfma(qa, B, sh_ld<CH>(sh.B[t.s][q]));
        A = A * qa;
      }
      // handed on here if the state is there already, else by the joining warp
      Vec<CH> v;
      const float* row = cut_row(a, t.k * kTile + cut, ch, v);
      const bool there = __all_sync(0xffffffffu, !row || is_full(v));
      if (there && ch < C) hand_state(a.states + (size_t)(a.t.n_nodes + t.k) * C + ch, vfma(A, v, B));
      if (lane == 0) sh.handed[t.s] = there;
      sh_st(sh.all[t.s][0], A);
      sh_st(sh.all[t.s][1], B);
    }
    warp_arrive(&sh.known[t.s]);
  }
}

// after: the states between tiles, which the forward left
template <int CH>
DEVI void bwd_publish(ScanShared& sh, ScanBack& back, const ScanWork& w, const float* after, int C,
                      int slab_ch, const WaitCtl& wc) {
  const int lane = threadIdx.x & 31;
  Tile t;
  for (int i = 0; next_tile(sh, sh.told, i, t, wc); ++i) {
    const int ch = t.slab * slab_ch + lane * CH;
    Vec<CH> h = ld_state_if(after + ((size_t)t.k * C - C) + ch, ch < C && (t.info & kInfoIn), Vec<CH>());
    if (!wait_phase(&sh.mapped[t.s], t.parity, wc)) return;
    if (t.info & kInfoMapped) {
#pragma unroll
      for (int q = 0; q < kScanWarps; ++q) {
        const Vec<CH> qb = sh_ld<CH>(sh.B[t.s][q]);
        sh_st(sh.B[t.s][q], h);
        h = vfma(sh_ld<CH>(sh.A[t.s][q]), h, qb);
      }
      Vec<CH> A = vec<CH>(1.f), R = vec<CH>(0.f);
#pragma unroll
      for (int q = kScanWarps - 1; q >= 0; --q) {
        const Vec<CH> qa = sh_ld<CH>(sh.A[t.s][q]), qr = sh_ld<CH>(back.R[t.s][q]);
        sh_st(sh.A[t.s][q], A);
        sh_st(back.R[t.s][q], R);
        R = vfma(qa, R, qr);
        A = A * qa;
      }
      if ((t.info & kInfoMap) && ch < C) hand_map(w.maps + ((size_t)t.k * C + ch) * 2, A, R);
      sh_st(sh.all[t.s][0], A);
      sh_st(sh.all[t.s][1], R);
    } else if (sh.cut[t.s] >= 0) {
      Vec<CH> R = vec<CH>(0.f);
      for (int q = sh.cut[t.s] / kWarpTokens; q >= 0; --q) R = vfma(sh_ld<CH>(sh.A[t.s][q]), R, sh_ld<CH>(back.R[t.s][q]));
      if (ch < C) hand_state(w.carry + (size_t)t.k * C + ch, R);
    }
    warp_arrive(&sh.known[t.s]);
  }
}

// A joining warp.  `dist` maps lie between the tile and the state it starts from.  FWD: that is the
// state behind the nearest tile before it that is no plain map or ends a group of kScanGroup; backward the same
// from the other side.  Groups bound the maps that a tile joins; within one, no tile waits for a state to be
// handed on.  rows: the states between tiles (backward: the gradients).
template <bool FWD, int CH, typename Late>
DEVI void scan_join(ScanShared& sh, const ScanWork& w, int C, float* rows, int slab_ch, int joiner, const Late& late,
                    const WaitCtl& wc) {
  const int lane = threadIdx.x & 31;
  Tile t;
  for (int i = joiner; next_tile(sh, sh.told, i, t, wc); i += kJoins) {
    const int info = t.info, ch = t.slab * slab_ch + lane * CH, dist = sh.dist[t.s];
    const bool on = ch < C, need = info & (FWD ? kInfoIn : kInfoOut);
    const int b = FWD ? t.k - 1 - dist : t.k + 1 + dist;
    const Joiner<CH> j{w, C, ch, b, FWD ? 1 : -1, dist, rows + (size_t)(need ? b : 0) * C + ch, on};
    Vec<CH> v = vec<CH>(0.f);
    if (FWD && sh.cut[t.s] >= 0) {
      if (!wait_phase(&sh.known[t.s], t.parity, wc)) return;
      if (!sh.handed[t.s]) {                           // what the publishing warp did not wait for
        bool ok = true;
        if constexpr (FWD) ok = late(t.k * kTile + sh.cut[t.s], ch, v);
        if (!ok) {
          if (lane == 0) sh.abort_flag = 1;
          return;
        }
        if (on) hand_state(rows + (size_t)t.k * C + ch, vfma(sh_ld<CH>(sh.all[t.s][0]), v, sh_ld<CH>(sh.all[t.s][1])));
      }
      v = vec<CH>(0.f);
    }
    if (need && !j.join(v, wc)) {
      if (lane == 0) sh.abort_flag = 1;
      return;
    }
    if (!wait_phase(&sh.known[t.s], t.parity, wc)) return;
    if ((info & kInfoMapped) && on)
      hand_state(rows + (size_t)t.k * C + ch, vfma(sh_ld<CH>(sh.all[t.s][0]), v, sh_ld<CH>(sh.all[t.s][1])));
    sh_st<CH>(sh.in[t.s], v);
    warp_arrive(&sh.ready[t.s]);
    warp_arrive(&sh.empty[t.s]);
  }
}

// The mapping warps, forward: a and b of every token, and the map of a warp's tokens.
template <typename T, int KIND>
DEVI void fwd_map(ScanShared& sh, uint8_t* slots, int warp, const WaitCtl& wc) {
  constexpr int CH = Lane<T>::CH;
  Tile t;
  for (int i = 0; next_tile(sh, sh.full, i, t, wc); ++i) {
    const Rows<T> rows(slots, t.s, warp);
    Vec<CH> A = vec<CH>(1.f), B = vec<CH>(0.f);
#pragma unroll 4
    for (int q = 0; q < kWarpTokens; ++q) {
      Vec<CH> a, b;
      token_of<KIND, sizeof(T) == 4>(rows.get(0, q), rows.get(1, q), a, b);
      rows.set_token(q, a, b);
      B = vfma(a, B, b);
      A = A * a;
    }
    const int cut = sh.cut[t.s] - warp * kWarpTokens;
    if ((unsigned)cut < (unsigned)kWarpTokens) {       // (rare: the map once more, from there)
      A = vec<CH>(1.f);
      B = vec<CH>(0.f);
#pragma unroll 1
      for (int q = cut; q < kWarpTokens; ++q) {
        const Vec<CH> a = rows.decay(q);
        B = rows.step(q, B);
        A = A * a;
      }
    }
    sh_st(sh.A[t.s][warp], A);
    sh_st(sh.B[t.s][warp], B);
    fence_proxy_async_smem();                          // a and b lie where the next copies go
    warp_arrive(&sh.mapped[t.s]);
  }
}

// Forward, the runs of a warp's 16 tokens between breaks and what is to be kept of them.  Loops are rolled: this
// is rare, and straight-line code for it would be fetched anew each time.
template <typename T>
struct FwdRuns {
  static constexpr int CH = Lane<T>::CH;
  const ScanFwd<T>& a;
  const Rows<T>& rows;
  ScanWalk& walk;
  ScanEnds& kept;
  int k, t0, ch;
  bool on;
  int serial;                              // the tile's number among those whose warps go one by one, 0: it is none
  // per lane q < 16: link of token t0 + q; its node if it is the node's last; its node; where in the tile the node that
  // it starts from ends, -1 if elsewhere
  int from, end, own, src;
  uint32_t breaks, ends, reset;            // a bit a token; reset: breaks that start from outside the tile
  DEVI uint32_t behind(int q) const { return q < 31 ? ~((2u << q) - 1u) : 0u; }
  DEVI int run_end(int q) const {
    const uint32_t m = breaks & behind(q);
    return m ? __ffs(m) - 1 : kWarpTokens;
  }
  // the tokens from q0 to the next break, h the state before them; returns the state behind them
  DEVI Vec<CH> run(Vec<CH> h, int q0) const {
    const int q1 = run_end(q0);
#pragma unroll 1
    while (q0 < q1) {
      const uint32_t m = ends >> q0;
      const int e = m ? q0 + __ffs(m) - 1 : kWarpTokens, stop = min(e + 1, q1);
      T* y = a.y + (size_t)(t0 + q0) * a.C + ch;
      const int rest = on ? a.t.N - t0 : 0;
#pragma unroll 4
      for (; q0 < stop; ++q0, y += a.C) {
        h = rows.step(q0, h);
        if (q0 < rest) *reinterpret_cast<uint32_t*>(y) = Lane<T>::pack(h);
      }
      if (e < q1) {                        // a node's last token: its state, for the user and for breaks
        const int n = __shfl_sync(0xffffffffu, end, e), tok = t0 + e - k * kTile, slot = tok / kKeep;
        if (on) hand_state(a.states + (size_t)n * a.C + ch, h);
        if (serial) {
          // no token's while it changes: whoever reads it looks at the token afterwards
          if ((threadIdx.x & 31) == 0) *(volatile int*)&kept.token[slot] = -1;
          __threadfence_block();
          __syncwarp();
          sh_st(kept.state[slot], h);
          __threadfence_block();
          __syncwarp();
          if ((threadIdx.x & 31) == 0) *(volatile int*)&kept.token[slot] = tok;
          row_written(walk, tok, serial);
        }
      }
    }
    return h;
  }
  // where the run that starts at token q begins, n its link
  DEVI const float* start_row(int q, int n) const {
    const int v = __shfl_sync(0xffffffffu, own, q);
    return n >= 0 ? a.states + (size_t)n * a.C : (a.init && n == kLinkRoot ? a.init + (size_t)v * a.C : nullptr);
  }
  // all initial states on their way at once
  DEVI void fetch_init() const {
    if (!a.init) return;
#pragma unroll 4
    for (int q = 0; q < kWarpTokens; ++q) {
      const int n = __shfl_sync(0xffffffffu, from, q), v = __shfl_sync(0xffffffffu, own, q);
      if (on && n == kLinkRoot) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.init + (size_t)v * a.C + ch));
    }
  }
  // Every token of the warp is such a run of its own (a step of many sequences: 4096 by 4096 channels in 103 us,
  // 187 run by run); h: the last one's state.
  DEVI bool single_runs(Vec<CH>& h, const WaitCtl& wc) const {
    bool ok = true;
    fetch_init();
#pragma unroll 1
    for (int g = 0; g < kWarpTokens && t0 + g < a.t.N; g += 4) {
      Vec<CH> s[4];
      int n[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        n[r] = __shfl_sync(0xffffffffu, from, g + r);
        const float* row = start_row(g + r, n[r]);
        s[r] = ld_state_if(row + ch, on && row, h);
      }
      T* y = a.y + (size_t)(t0 + g) * a.C + ch;
#pragma unroll
      for (int r = 0; r < 4; ++r, y += a.C) {
        if (t0 + g + r >= a.t.N) break;
        ok = arrived(a.states + (size_t)n[r] * a.C + ch, s[r], on && n[r] >= 0, wc, a.w.ctl + 2) && ok;
        h = rows.step(g + r, s[r]);
        const int e = __shfl_sync(0xffffffffu, end, g + r);
        if (on) {
          *reinterpret_cast<uint32_t*>(y) = Lane<T>::pack(h);
          if (e >= 0) hand_state(a.states + (size_t)e * a.C + ch, h);
        }
      }
    }
    return __all_sync(0xffffffffu, ok);
  }
  // All runs that start from outside the tile, which wait for nothing in it.  `known`: the last run is one of them,
  // whose end is then the state behind the warp.  False if a wait gave up.
  DEVI bool known_runs(Vec<CH>& last, bool& known, const WaitCtl& wc) const {
    if (reset && !serial && reset == (1u << min(kWarpTokens, a.t.N - t0)) - 1u) {
      known = true;
      return single_runs(last, wc);
    }
#pragma unroll 1
    for (uint32_t m = reset; m;) {
      // the starts of four runs at a time: their loads are in flight together
      Vec<CH> s[4];
      int q[4], n[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        q[r] = m ? __ffs(m) - 1 : -1;
        m &= m - 1;
        n[r] = __shfl_sync(0xffffffffu, from, max(q[r], 0));
        const float* row = start_row(max(q[r], 0), n[r]);
        s[r] = ld_state_if(row + ch, on && row && q[r] >= 0, last);
      }
#pragma unroll 1
      for (int r = 0; r < 4; ++r) {
        if (q[0] < 0) break;
        const bool ok = arrived(a.states + (size_t)n[0] * a.C + ch, s[0], on && n[0] >= 0, wc, a.w.ctl + 2);
        if (!__all_sync(0xffffffffu, ok)) return false;
        last = run(s[0], q[0]);
        s[0] = s[1]; s[1] = s[2]; s[2] = s[3];
        q[0] = q[1]; q[1] = q[2]; q[2] = q[3]; q[3] = -1;
        n[0] = n[1]; n[1] = n[2]; n[2] = n[3];
      }
    }
    known = reset && (breaks >> (31 - __clz(reset))) == 1u;
    return true;
  }
  // The runs that wait: the one that comes into the warp, and those that start from nodes of this tile.  v: the
  // state behind the last of them; false if a wait gave up.
  DEVI bool waiting_runs(Vec<CH> h, Vec<CH>& v, const WaitCtl& wc) const {
    if (!(breaks & 1u)) h = run(h, 0);
#pragma unroll 1
    for (uint32_t m = breaks & ~reset; m; m &= m - 1) {
      const int q = __ffs(m) - 1, n = __shfl_sync(0xffffffffu, from, q);
      const int tok = __shfl_sync(0xffffffffu, src, q), slot = tok / kKeep;
      const bool ok = wait_until([&] { return *(volatile int*)&walk.row_of[tok] == serial; }, wc, a.w.ctl + 2);
      if (!__all_sync(0xffffffffu, ok)) return false;
      __threadfence_block();
      // kept, unless the end of another node within the same tokens has taken its place (looked at twice: the
      // other one may come meanwhile)
      const Vec<CH> near = sh_ld<CH>(kept.state[slot]);
      __threadfence_block();
      const bool here = __all_sync(0xffffffffu, *(volatile int*)&kept.token[slot] == tok);
      h = here ? near : ld_state_if(a.states + (size_t)n * a.C + ch, on, h);
      h = run(h, q);
    }
    v = h;
    return true;
  }
};

// The walking warps, forward.  Returns where a wait gave up or the tiles have ended.
template <typename T>
DEVI void fwd_walk(const ScanFwd<T>& a, ScanShared& sh, ScanWalk& g, ScanEnds& kept, uint8_t* slots,
                   int warp, const WaitCtl& wc) {
  constexpr int CH = Lane<T>::CH, SLAB = kRow / (int)sizeof(T);
  const int lane = threadIdx.x & 31;
  uint32_t n_own = 0;                                  // uses of the walking warps' barriers so far
  int n_turn = 0;
  Tile t;
  for (int i = 0; next_tile(sh, sh.told, i, t, wc); ++i) {
    const Rows<T> rows(slots, t.s, warp);
    const int ch = t.slab * SLAB + lane * CH;          // the lane's first channel
    const int t0 = t.k * kTile + warp * kWarpTokens;
    const bool serial = t.info & kInfoSerial;
    n_turn += serial;
    FwdRuns<T> f{a, rows, g, kept, t.k, t0, ch, ch < a.C, serial ? n_turn : 0, kLinkChain, -1, 0, -1, 0u, 0u, 0u};
    const bool special = t.info & (kInfoBreak | kInfoEnd);
    if (special) {
      if (lane < kWarpTokens && t0 + lane < a.t.N) {
        f.from = a.w.link[t0 + lane];
        f.end = a.w.end[t0 + lane];
        f.own = a.t.tok_node[t0 + lane];
        if (f.from >= 0) {
          const int at = a.t.tok_start[f.from] + a.t.node_len[f.from] - 1;
          if (at / kTile == t.k) f.src = at % kTile;
        }
      }
      f.breaks = __ballot_sync(0xffffffffu, f.from != kLinkChain);
      f.ends = __ballot_sync(0xffffffffu, f.end >= 0);
      f.reset = f.breaks & ~__ballot_sync(0xffffffffu, f.src >= 0);
    }
    Vec<CH> last = vec<CH>(0.f);                       // the state behind the warp
    bool last_known = false;
    if (t.info & kInfoBreak) {
      if (!wait_phase(&sh.known[t.s], t.parity, wc)) return;
      if (serial) {                                    // no warp is a tile ahead, where its turn would overtake this one's
        warp_arrive(&g.own);
        if (!wait_phase(&g.own, n_own & 1, wc)) return;
        ++n_own;
      }
      if (!f.known_runs(last, last_known, wc)) {
        if (lane == 0) sh.abort_flag = 1;
        return;
      }
      if (!serial) {                                   // every warp's map is there
        if (f.breaks) sh_st(sh.B[t.s][warp], last);
        if (lane == 0) sh.reset[t.s][warp] = f.breaks != 0;
        warp_arrive(&g.own);
        if (!wait_phase(&g.own, n_own & 1, wc)) return;
        ++n_own;
      }
    }
    // The state before the warp: from the maps of the warps before it; where a break starts from a node that
    // ends in this very tile, from the warp before it, which has then kept its nodes' states.
    auto past = [&](int q, Vec<CH> v) {                // the state behind warp q's tokens, by their map
      return vfma(sh_ld<CH>(sh.A[t.s][q]), v, sh_ld<CH>(sh.B[t.s][q]));
    };
    auto hand_on = [&](Vec<CH> v) {                    // to the warps and the tiles behind
      if (serial && warp < kScanWarps - 1) {
        sh_st(g.carry[warp], v);
        warp_arrive(&g.turn[warp + 1]);
      }
      if (warp == kScanWarps - 1 && f.on && sh.cut[t.s] < 0) hand_state(a.states + (size_t)(a.t.n_nodes + t.k) * a.C + ch, v);
    };
    if (last_known) hand_on(last);
    Vec<CH> h = vec<CH>(0.f);
    if (f.breaks & 1u) {
      // nothing comes into the warp (a turn that it does not take is over when the warps meet in the next such tile)
    } else if (!wait_phase(&sh.ready[t.s], t.parity, wc)) {
      return;
    } else if (t.info & kInfoMapped) {
      h = sh_ld<CH>(sh.in[t.s]);
      h = vfma(sh_ld<CH>(sh.A[t.s][warp]), h, sh_ld<CH>(sh.B[t.s][warp]));
    } else if (!serial) {
      h = sh_ld<CH>(sh.in[t.s]);
      for (int q = 0; q < warp; ++q) h = sh.reset[t.s][q] ? sh_ld<CH>(sh.B[t.s][q]) : past(q, h);
    } else if (warp == 0) {
      h = sh_ld<CH>(sh.in[t.s]);
    } else {
      if (!wait_phase(&g.turn[warp], (n_turn - 1) & 1, wc)) return;
      h = sh_ld<CH>(g.carry[warp - 1]);
    }
    // a warp without breaks hands on by its maps, before it walks
    if ((t.info & kInfoBreak) && !f.breaks) hand_on(past(warp, h));
    if (f.breaks || f.ends) {
      Vec<CH> v;
      if (!f.waiting_runs(h, v, wc)) {
        if (lane == 0) sh.abort_flag = 1;
        return;
      }
      if (f.breaks && !last_known) hand_on(v);
    } else {
      T* y = a.y + (size_t)t0 * a.C + ch;
      const int rest = f.on ? a.t.N - t0 : 0;          // tokens to write
#pragma unroll 4
      for (int q = 0; q < kWarpTokens; ++q, y += a.C) {
        h = rows.step(q, h);
        if (q < rest) *reinterpret_cast<uint32_t*>(y) = Lane<T>::pack(h);
      }
    }
    warp_arrive(&sh.empty[t.s]);
  }
}

// The mapping warps, backward: p, and a warp's maps of h and of the gradient (which share the factor).
template <typename T, int KIND>
DEVI void bwd_map(ScanShared& sh, ScanBack& back, uint8_t* slots, int warp, const WaitCtl& wc) {
  constexpr int CH = Lane<T>::CH;
  Tile t;
  for (int i = 0; next_tile(sh, sh.full, i, t, wc); ++i) {
    const Rows<T> rows(slots, t.s, warp);
    int cut = sh.cut[t.s] - warp * kWarpTokens;        // what the warp hands on comes from the tokens before it
    if ((unsigned)cut >= (unsigned)kWarpTokens) cut = kWarpTokens;
    Vec<CH> A = vec<CH>(1.f), B = vec<CH>(0.f), R = vec<CH>(0.f);
#pragma unroll 4
    for (int q = 0; q < kWarpTokens; ++q) {
      const Vec<CH> p = gate_of<KIND>(rows.get(0, q));
      rows.set_p(q, p);
      B = advance<KIND>(p, rows.get(1, q), B);
      // the gradient's map, from the first token on: u before = R + A u behind
      if (q < cut) {
        A = decayed(p, A);
        R = vfma(A, rows.get(2, q), R);
      }
    }
    sh_st(sh.A[t.s][warp], A);
    sh_st(sh.B[t.s][warp], B);
    sh_st(back.R[t.s][warp], R);
    fence_proxy_async_smem();
    warp_arrive(&sh.mapped[t.s]);
  }
}

// Backward, a warp at whose 16 tokens paths break or join.  One token at a time, in rolled loops: it is rare, and
// straight-line code for four tokens (some 10 KB) was fetched anew each time, which took longer than the steps.
template <typename T, int KIND>
struct BwdBreaks {
  static constexpr int CH = Lane<T>::CH;
  const ScanBwd<T>& a;
  const Rows<T>& rows;
  int t0, ch;
  bool on;
  int from, end, kid, sib, own;            // per lane q < 16, of token t0 + q; own: its node
  uint32_t breaks, joins;
  int kid_at, sib_at;                      // per lane: the token of this tile at which kid, sib starts; -1: in another
  // the state that the break at token q starts from
  DEVI Vec<CH> start_of(int q) const {
    const int n = __shfl_sync(0xffffffffu, from, q), v = __shfl_sync(0xffffffffu, own, q);
    const float* row = n >= 0 ? a.states + (size_t)n * a.C : (a.init ? a.init + (size_t)v * a.C : nullptr);
    return ld_given_if(row + ch, on && row, Vec<CH>());
  }
  // h before token q, from h before token g; held: the state that the break at token `at` starts from
  DEVI Vec<CH> before(int g, int q, Vec<CH> h, int& at, Vec<CH>& held) const {
    const uint32_t m = breaks & ((2u << q) - 1u) & ~((1u << g) - 1u);
    int r = g;
    if (m) {
      r = 31 - __clz(m);
      if (r != at) held = start_of(r);
      at = r;
      h = held;
    }
#pragma unroll 1
    for (; r < q; ++r) h = advance<KIND>(rows.p(r), rows.get(1, r), h);
    return h;
  }
  // dy of token q and what joins it: kid: the next node that starts from this one's state, with those behind it;
  // end: the node's own final state.  False if a wait gave up.
  DEVI bool sum(int q, Vec<CH>& d, const WaitCtl& wc) const {
    d = rows.get(2, q);
    if (!((joins >> q) & 1u)) return true;
    const int kd = __shfl_sync(0xffffffffu, kid, q), e = __shfl_sync(0xffffffffu, end, q);
    const float* row = a.w.dnode + (size_t)kd * a.C + ch;
    const Vec<CH> f = ld_state_if(a.d_final + (size_t)e * a.C + ch, on && a.d_final && e >= 0, d);
    Vec<CH> k = ld_state_if(row, on && kd >= 0, d);
    const bool ok = arrived(row, k, on && kd >= 0, wc, a.w.ctl + 2);
    d = d + (f + k);
    return __all_sync(0xffffffffu, ok);
  }
};

// The walking warps, backward: h before every token, then the gradients from the last token to the first.
template <typename T, int KIND>
DEVI void bwd_walk(const ScanBwd<T>& a, ScanShared& sh, ScanBack& back, ScanWalk& gr, uint8_t* slots,
                   int warp, const WaitCtl& wc) {
  constexpr int CH = Lane<T>::CH, SLAB = kRow / (int)sizeof(T);
  const int lane = threadIdx.x & 31;
  uint32_t n_own = 0;
  int n_turn = 0;
  Tile t;
  for (int i = 0; next_tile(sh, sh.told, i, t, wc); ++i) {
    const Rows<T> rows(slots, t.s, warp);
    const int ch = t.slab * SLAB + lane * CH;
    const int t0 = t.k * kTile + warp * kWarpTokens;
    const bool mapped = t.info & kInfoMapped, serial = t.info & kInfoSerialBack;
    BwdBreaks<T, KIND> f{a, rows, t0, ch, ch < a.C, kLinkChain, -1, -1, -1, -1, 0u, 0u, -1, -1};
    n_turn += serial;
    const bool on = f.on;
    Vec<CH> h = vec<CH>(0.f);
    if (!mapped) {
      h = ld_state_if(a.states + (size_t)(a.t.n_nodes + t.k - 1) * a.C + ch, on && (t.info & kInfoIn), h);
      if (lane < kWarpTokens && t0 + lane < a.t.N) {
        const int j = t0 + lane;
        f.from = a.w.link[j];
        f.end = a.w.end[j];
        f.kid = a.w.kid[j];
        f.sib = a.w.sib[j];
        f.own = a.t.tok_node[j];
        // (a kid or sib in this tile: its first token there)
        if (f.kid >= 0 && a.t.tok_start[f.kid] / kTile == t.k) f.kid_at = a.t.tok_start[f.kid] - t.k * kTile;
        if (f.sib >= 0 && a.t.tok_start[f.sib] / kTile == t.k) f.sib_at = a.t.tok_start[f.sib] - t.k * kTile;
      }
      f.breaks = __ballot_sync(0xffffffffu, f.from != kLinkChain);
      f.joins = __ballot_sync(0xffffffffu, f.kid >= 0 || (f.end >= 0 && a.d_final));
    }
    const uint32_t special = f.breaks | f.joins;
    // Up to the four tokens in which the warp's first break lies h depends on what comes into the warp, and what the
    // warp hands on depends on the tokens before that break only; in some of these (`late`) a node of this tile joins.
    const int first = f.breaks ? __ffs(f.breaks) - 1 : kWarpTokens, known = min(first, kWarpTokens - 1) & ~3;
    const uint32_t kids = __ballot_sync(0xffffffffu, f.kid_at >= 0);
    const bool late = kids & ((1u << first) - 1u);
    if (!wait_phase(&sh.known[t.s], t.parity, wc)) return;
    bool ok = true;
    if (!mapped) {
      if (f.breaks) {                                  // h behind the warp does not depend on h before it
        Vec<CH> v = vec<CH>(0.f);
#pragma unroll 1
        for (int q = first; q < kWarpTokens; ++q) {
          if (q > first && q % 4 == 0) sh_st(back.before[warp][q / 4], v);
          if ((f.breaks >> q) & 1u) v = f.start_of(q);
          v = advance<KIND>(rows.p(q), rows.get(1, q), v);
        }
        sh_st(sh.B[t.s][warp], v);
      }
      if (special && !late) {
        Vec<CH> R = vec<CH>(0.f), d;
#pragma unroll 1
        for (int q = first - 1; q >= 0; --q) {
          ok = f.sum(q, d, wc) && ok;
          R = decayed(rows.p(q), d + R);
        }
        sh_st(back.R[t.s][warp], R);
      }
      if (lane == 0) sh.reset[t.s][warp] = f.breaks != 0;
      warp_arrive(&gr.own);
      if (!wait_phase(&gr.own, n_own & 1, wc)) return;
      ++n_own;
    }
    if (mapped) {
      h = sh_ld<CH>(sh.B[t.s][warp]);
    } else {
      for (int q = 0; q < warp; ++q) {
        const Vec<CH> qb = sh_ld<CH>(sh.B[t.s][q]);
        h = sh.reset[t.s][q] ? qb : vfma(sh_ld<CH>(sh.A[t.s][q]), h, qb);
      }
    }
    // h before every fourth token; the others are stepped to again on the way back (16 values a lane would stay in
    // registers only in straight-line code of 15 KB, which the warps' other code would push out of the cache)
#pragma unroll 1
    for (int g = 0; g < known; g += 4) {
      sh_st(back.before[warp][g / 4], h);
#pragma unroll
      for (int q = 0; q < 4; ++q) h = advance<KIND>(rows.p(g + q), rows.get(1, g + q), h);
    }
    sh_st(back.before[warp][known / 4], h);
    // the gradient behind the warp, as the state before it in the forward
    auto hand_on = [&](Vec<CH> v) {                    // to the warps and the tiles before
      if (serial && warp > 0) {
        sh_st(gr.carry[warp], v);
        warp_arrive(&gr.turn[warp - 1]);
      }
      if (warp == 0 && on && sh.cut[t.s] < 0) hand_state(a.w.carry + (size_t)t.k * a.C + ch, v);
    };
    if (f.breaks && !late) hand_on(sh_ld<CH>(back.R[t.s][warp]));
    if (!wait_phase(&sh.ready[t.s], t.parity, wc)) return;
    Vec<CH> u = sh_ld<CH>(sh.in[t.s]);
    if (mapped) {
      u = vfma(sh_ld<CH>(sh.A[t.s][warp]), u, sh_ld<CH>(back.R[t.s][warp]));
    } else if (!serial) {
      for (int q = kScanWarps - 1; q > warp; --q) {
        const Vec<CH> qr = sh_ld<CH>(back.R[t.s][q]);
        u = sh.reset[t.s][q] ? qr : vfma(sh_ld<CH>(sh.A[t.s][q]), u, qr);
      }
    } else if (warp < kScanWarps - 1) {
      if (!wait_phase(&gr.turn[warp], (n_turn - 1) & 1, wc)) return;
      u = sh_ld<CH>(gr.carry[warp + 1]);
    }
    // a warp in which nothing of this tile joins hands on by its map, before it walks
    if (!mapped && !f.breaks && !late) hand_on(vfma(sh_ld<CH>(sh.A[t.s][warp]), u, sh_ld<CH>(back.R[t.s][warp])));
    auto wait_row = [&](int tok) {                     // of a node that starts in this tile
      const bool there = wait_until([&] { return *(volatile int*)&gr.row_of[tok] == n_turn; }, wc, a.w.ctl + 2);
      ok = __all_sync(0xffffffffu, there) && ok;
      __threadfence_block();
    };
    // token q: lam = what reaches it; its gradients; u before it
    auto step = [&](int q, Vec<CH> lam, Vec<CH> before) {
      const Vec<CH> p = rows.p(q);
      Vec<CH> dx, dg;
      if (KIND == TREE_GATE_SIGMOID) {
        Vec<CH> m, n;                                  // the smaller of a and 1 - a: m; lam by it, and by the larger
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          m.v[c] = fabsf(p.v[c]);
          n.v[c] = -m.v[c];
        }
        const Vec<CH> v = m * lam, w = vfma(n, lam, lam);
        u = pick(p, w, v);
        dx = pick(p, v, w);
        dg = vfma(n, v, v) * (before - rows.get(1, q));
      } else {
        u = decayed(p, lam);
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
    if (!special) {
#pragma unroll 1
      for (int g = kWarpTokens - 4; g >= 0; g -= 4) {
        Vec<CH> b[4];
        b[0] = sh_ld<CH>(back.before[warp][g / 4]);
#pragma unroll
        for (int q = 0; q < 3; ++q) b[q + 1] = advance<KIND>(rows.p(g + q), rows.get(1, g + q), b[q]);
#pragma unroll
        for (int q = 3; q >= 0; --q) step(g + q, rows.get(2, g + q) + u, b[q]);
      }
    } else
#pragma unroll 1
    for (int g = kWarpTokens - 4; g >= 0; g -= 4) {
      Vec<CH> b[4];
      h = sh_ld<CH>(back.before[warp][g / 4]);
      if (!((special >> g) & 15u)) {
        b[0] = h;
#pragma unroll
        for (int q = 0; q < 3; ++q) b[q + 1] = advance<KIND>(rows.p(g + q), rows.get(1, g + q), b[q]);
#pragma unroll
        for (int q = 3; q >= 0; --q) step(g + q, rows.get(2, g + q) + u, b[q]);
      } else {
        int held_at = -1;
        Vec<CH> held = h;
#pragma unroll 1
        for (int q = g + 3; q >= g; --q) {
          const int kid_at = __shfl_sync(0xffffffffu, f.kid_at, q);
          if (kid_at >= 0) wait_row(kid_at);
          Vec<CH> d;
          ok = f.sum(q, d, wc) && ok;
          step(q, d + u, f.before(g, q, h, held_at, held));
          if (!((f.breaks >> q) & 1u)) continue;
          // what this path hands to the state it started from
          const int n = __shfl_sync(0xffffffffu, f.from, q), v = __shfl_sync(0xffffffffu, f.own, q);
          const int sb = __shfl_sync(0xffffffffu, f.sib, q), sib_at = __shfl_sync(0xffffffffu, f.sib_at, q);
          if (sib_at >= 0) wait_row(sib_at);
          const float* row = a.w.dnode + (size_t)sb * a.C + ch;
          Vec<CH> later = ld_state_if(row, on && sb >= 0, u);
          ok = __all_sync(0xffffffffu, arrived(row, later, on && sb >= 0, wc, a.w.ctl + 2)) && ok;
          if (on && n >= 0) hand_state(a.w.dnode + (size_t)v * a.C + ch, u + later);
          if (on && n == kLinkRoot && a.d_init) st_state(a.d_init + (size_t)v * a.C + ch, u);
          u = vec<CH>(0.f);
          if (serial) row_written(gr, warp * kWarpTokens + q, n_turn);
        }
      }
    }
    if (!ok) {
      if (lane == 0) sh.abort_flag = 1;
      return;
    }
    if (late) hand_on(u);
    warp_arrive(&sh.empty[t.s]);
  }
}

constexpr int scan_smem(int slots) { return slots * kPlanes * kPlane + 128; }

DEVI uint8_t* scan_align(uint8_t* p) { return p + ((128u - (smem_u32(p) & 127u)) & 127u); }   // copies land on 128 bytes

DEVI void scan_init(ScanShared& sh, ScanWalk& walk) {
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&sh.full[s], 1);
      mbar_init(&sh.told[s], 1);
      mbar_init(&sh.mapped[s], kScanWarps);
      mbar_init(&sh.known[s], 1);
      mbar_init(&sh.ready[s], 1);
      mbar_init(&sh.empty[s], kScanWarps + 1);     // the walking warps and the joining warp
    }
    for (int q = 0; q < kTile; ++q) walk.row_of[q] = 0;
    mbar_init(&walk.own, kScanWarps);
    for (int q = 0; q < kScanWarps; ++q) mbar_init(&walk.turn[q], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
}

// Every wait between warps is on an mbarrier and has a limit; the first that gives up raises the block's
// abort flag, which ends the others.
template <typename T, int KIND>
__global__ void __launch_bounds__(kScanThreads, 1) k_scan_fwd(const __grid_constant__ CUtensorMap tm_gate,
                                                              const __grid_constant__ CUtensorMap tm_x,
                                                              const ScanFwd<T> a) {
  constexpr int CH = Lane<T>::CH, SLAB = kRow / (int)sizeof(T);
  extern __shared__ uint8_t smem_raw[];
  __shared__ ScanShared sh;
  __shared__ ScanWalk walk;
  __shared__ ScanEnds kept;
  uint8_t* slots = scan_align(smem_raw);
  scan_init(sh, walk);
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  constexpr int WALK = kScanWarps, LOAD = 2 * kScanWarps;     // first warp of each role
  const int warp = threadIdx.x >> 5;
  if (warp < WALK) {
    fwd_map<T, KIND>(sh, slots, warp, wc);
  } else if (warp < LOAD) {
    fwd_walk<T>(a, sh, walk, kept, slots, warp - WALK, wc);
  } else if (warp == LOAD) {
    const CUtensorMap* tm[2] = {&tm_gate, &tm_x};
    scan_load<true>(sh, slots, tm, a.w, a.t.n_tiles, a.slabs, SLAB, false, wc);
  } else if (warp == LOAD + 1) {
    fwd_publish(a, sh, SLAB, wc);
  } else {
    auto late = [&](int j, int ch, Vec<CH>& v) {
      const float* row = cut_row(a, j, ch, v);
      return __all_sync(0xffffffffu, arrived(row, v, row != nullptr, wc, a.w.ctl + 2)) != 0;
    };
    scan_join<true, CH>(sh, a.w, a.C, a.states + (size_t)a.t.n_nodes * a.C, SLAB,
                                   warp - LOAD - 2, late, wc);
  }
}

template <typename T, int KIND>
__global__ void __launch_bounds__(kScanThreads, 1) k_scan_bwd(const __grid_constant__ CUtensorMap tm_gate,
                                                              const __grid_constant__ CUtensorMap tm_x,
                                                              const __grid_constant__ CUtensorMap tm_dy,
                                                              const ScanBwd<T> a) {
  constexpr int CH = Lane<T>::CH, SLAB = kRow / (int)sizeof(T);
  extern __shared__ uint8_t smem_raw[];
  __shared__ ScanShared sh;
  __shared__ ScanBack back;
  __shared__ ScanWalk walk;
  uint8_t* slots = scan_align(smem_raw);
  scan_init(sh, walk);
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  constexpr int WALK = kScanWarps, LOAD = 2 * kScanWarps;     // first warp of each role
  const int warp = threadIdx.x >> 5;
  if (warp < WALK) {
    bwd_map<T, KIND>(sh, back, slots, warp, wc);
  } else if (warp < LOAD) {
    bwd_walk<T, KIND>(a, sh, back, walk, slots, warp - WALK, wc);
  } else if (warp == LOAD) {
    const CUtensorMap* tm[3] = {&tm_gate, &tm_x, &tm_dy};
    scan_load<false>(sh, slots, tm, a.w, a.t.n_tiles, a.slabs, SLAB, a.d_final != nullptr, wc);
  } else if (warp == LOAD + 1) {
    bwd_publish<CH>(sh, back, a.w, a.states + (size_t)a.t.n_nodes * a.C, a.C, SLAB, wc);
  } else {
    scan_join<false, CH>(sh, a.w, a.C, a.w.carry, SLAB,
                                    warp - LOAD - 2, 0, wc);
  }
}

// Forward for a step of decoding: one launch, no maps and nothing to wait for.  A block takes a slab and up to
// kStepMost tokens.  Either these are all there are, of whatever tree; or every node is a sequence of its own,
// most of one token and none of many, and the block walks those that begin in it.  Latency is all: the gates and inputs of a warp's
// eight tokens are on their way while lanes 0-7 find out where these start from; then each warp walks the trees
// that begin within its eight tokens to their ends.  By 4096 bf16 channels, in us (by the kernels for many tokens):
// 64 one-token nodes 4.6 (20.6), 300 6.7 (27), 4096 57 (104); a chain of 256 11.2 (11.3), one of 128 with 128
// one-token children 26 (28).  A sequence among one-token nodes is walked by one warp a slab, behind its block's tokens
// from memory: 300 nodes and one of 128 tokens 14 (26), of 192 21 (26), of 256 29 (26), of 4096 649 (53); 4096 nodes and
// one of 128 53 (83), of 512 105 (84).  Above kStepLongest that is left to the others.
constexpr int kStepTokens = 8, kStepMost = 2 * kTile;  // a warp's tokens; a block's (1024 threads)
constexpr int kStepLongest = kTile;
template <typename T>
constexpr int step_smem(int n) { return (n + kStepTokens - 1) / kStepTokens * kStepTokens * 2 * 32 * Lane<T>::CH * 4; }

template <typename T, int KIND>
__global__ void __launch_bounds__(32 * kStepMost / kStepTokens) k_scan_step(const T* gate, const T* x, int span, const ScanFwd<T> a) {
  constexpr int CH = Lane<T>::CH, SLAB = kRow / (int)sizeof(T);
  extern __shared__ float step_rows[];                 // per token: its decays, its inputs (its states once walked)
  __shared__ int from[kStepMost], node[kStepMost];     // where a break's state lies, the token's node
  __shared__ uint32_t bits[kStepMost / kStepTokens][3];             // per warp's tokens: roots' first, breaks, nodes' last
  const int base = blockIdx.y * span, n = min(span, a.t.N - base);  // the block's tokens: counted from base below
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ch = blockIdx.x * SLAB + lane * CH, t0 = warp * kStepTokens, j = t0 + lane;
  const bool on = ch < a.C;
  auto decay = [&](int q) { return step_rows + q * 2 * 32 * CH; };
  auto input = [&](int q) { return step_rows + (q * 2 + 1) * 32 * CH; };
  auto word = [&](const T* p, int q) { return __ldg(reinterpret_cast<const uint32_t*>(p + (size_t)(base + q) * a.C + ch)); };
  // behind token q, h the state there: kept between tiles; nothing goes on from the last token's tile, whose row holds
  // no leftovers
  auto between = [&](int q, Vec<CH> h) {
    const int t = base + q + 1;
    if (on && t == a.t.N) st_state(a.states + (size_t)(a.t.n_nodes + (t - 1) / kTile) * a.C + ch, t % kTile ? vec<CH>(0.f) : h);
    else if (on && t % kTile == 0) st_state(a.states + (size_t)(a.t.n_nodes + (t - 1) / kTile) * a.C + ch, h);
  };
  uint32_t gw[kStepTokens], xw[kStepTokens];
#pragma unroll
  for (int q = 0; q < kStepTokens; ++q) {
    const bool in = on && t0 + q < n;
    gw[q] = in ? word(gate, t0 + q) : 0u;
    xw[q] = in ? word(x, t0 + q) : 0u;
  }
  int start = kLinkChain, own = 0;
  bool last = false;
  if (lane < kStepTokens && j < n) {
    own = a.t.tok_node[base + j];
    const int first = a.t.tok_start[own] - base, len = a.t.node_len[own];
    const int up = j == first ? scan_token_ancestor(own, a.t) : -1;
    const int src = up < 0 ? -1 : a.t.tok_start[up] + a.t.node_len[up] - 1 - base;
    if (j == first) start = src < 0 || src >= j ? kLinkRoot : src == j - 1 ? kLinkChain : up;
    last = j == first + len - 1;
    from[j] = src;
    node[j] = own;
  }
  const uint32_t roots = __ballot_sync(0xffffffffu, start == kLinkRoot);
  const uint32_t breaks = __ballot_sync(0xffffffffu, start != kLinkChain), ends = __ballot_sync(0xffffffffu, last);
  if (lane == 0) {
    bits[warp][0] = roots;
    bits[warp][1] = breaks;
    bits[warp][2] = ends;
  }
  // a root's input takes its initial state in: h = a init + b
  Vec<CH> h0[kStepTokens];
#pragma unroll
  for (int q = 0; q < kStepTokens; ++q) {
    const int v = __shfl_sync(0xffffffffu, own, q);
    h0[q] = ld_state_if(a.init + (size_t)v * a.C + ch, on && a.init && ((roots >> q) & 1u), vec<CH>(0.f));
  }
#pragma unroll
  for (int q = 0; q < kStepTokens; ++q) {
    if (t0 + q >= n) break;
    Vec<CH> d, b;
    token_of<KIND, sizeof(T) == 4>(Lane<T>::unpack(gw[q]), Lane<T>::unpack(xw[q]), d, b);
    if ((roots >> q) & 1u) b = vfma(d, h0[q], b);
    sh_st(decay(t0 + q), d);
    sh_st(input(t0 + q), b);
  }
  // rows of nodes without tokens
  for (int v0 = blockIdx.y * blockDim.x + warp * 32; v0 < a.t.n_nodes; v0 += gridDim.y * blockDim.x) {
    const int v = v0 + lane;
    uint32_t m = __ballot_sync(0xffffffffu, v < a.t.n_nodes && a.t.node_len[min(v, a.t.n_nodes - 1)] <= 0);
    for (; m; m &= m - 1)
      if (on) st_state(a.states + (size_t)(v0 + __ffs(m) - 1) * a.C + ch, vec<CH>(0.f));
  }
  __syncthreads();
  if (!roots) return;
  Vec<CH> h = vec<CH>(0.f);
  int q0 = __ffs(roots) - 1;
#pragma unroll 1
  for (int w = warp; w * kStepTokens < n; ++w, q0 = 0) {
    const uint32_t rt = bits[w][0], br = bits[w][1], en = bits[w][2];
    const int at = w * kStepTokens, q1 = min(w > warp && rt ? __ffs(rt) - 1 : kStepTokens, n - at);
    Vec<CH> d[kStepTokens], b[kStepTokens];
    int src[kStepTokens];
#pragma unroll
    for (int q = 0; q < kStepTokens; ++q) {
      d[q] = sh_ld<CH>(decay(at + q));
      b[q] = sh_ld<CH>(input(at + q));
      src[q] = from[at + q];
    }
    T* y = a.y + (size_t)(base + at) * a.C + ch;
    if (!br && q1 == kStepTokens) {                    // (no branch between the tokens: a chain of 128 by 4096 in 6.9 us, else 13.3)
#pragma unroll
      for (int q = 0; q < kStepTokens; ++q, y += a.C) {
        h = vfma(d[q], h, b[q]);
        b[q] = h;
        if (on) *reinterpret_cast<uint32_t*>(y) = Lane<T>::pack(h);
      }
#pragma unroll
      for (int q = 0; q < kStepTokens; ++q) sh_st(input(at + q), b[q]);
    } else {
#pragma unroll
      for (int q = 0; q < kStepTokens; ++q, y += a.C) {
        if (q < q0 || q >= q1) continue;
        if ((br >> q) & 1u) h = (rt >> q) & 1u ? vec<CH>(0.f) : sh_ld<CH>(input(src[q]));
        h = vfma(d[q], h, b[q]);
        sh_st(input(at + q), h);
        if (on) *reinterpret_cast<uint32_t*>(y) = Lane<T>::pack(h);
      }
    }
    for (uint32_t m = en & ~((1u << q0) - 1u) & ((1u << q1) - 1u); m; m &= m - 1) {
      const int q = at + __ffs(m) - 1;
      if (on) st_state(a.states + (size_t)node[q] * a.C + ch, sh_ld<CH>(input(q)));
    }
    if (w > warp && rt) return;
    between(min(at + kStepTokens, n) - 1, h);
  }
  // a sequence that goes on behind the block's tokens (only where every node is a sequence of its own)
  if (base + n >= a.t.N) return;
  const int v = node[n - 1], end = min(a.t.tok_start[v] + a.t.node_len[v], a.t.N) - base;
#pragma unroll 1
  for (int at = n; at < end; at += kStepTokens) {
#pragma unroll
    for (int q = 0; q < kStepTokens; ++q) {
      const bool in = on && at + q < end;
      gw[q] = in ? word(gate, at + q) : 0u;
      xw[q] = in ? word(x, at + q) : 0u;
    }
#pragma unroll
    for (int q = 0; q < kStepTokens; ++q) {
      if (at + q >= end) break;
      Vec<CH> d, b;
      token_of<KIND, sizeof(T) == 4>(Lane<T>::unpack(gw[q]), Lane<T>::unpack(xw[q]), d, b);
      h = vfma(d, h, b);
      if (on) *reinterpret_cast<uint32_t*>(a.y + (size_t)(base + at + q) * a.C + ch) = Lane<T>::pack(h);
      if (on && at + q == end - 1) st_state(a.states + (size_t)v * a.C + ch, h);
      between(at + q, h);
    }
  }
}

// ---------------------------------------------------------------------------------------------
// host side

int scan_tiles(const tree_plan_t* p) { return (int)(((int64_t)p->n_tokens + kTile - 1) / kTile); }

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// slabs of 128 bytes of channels: counted for the narrower type, which has the more of them
int scan_slabs(int C, int dtype) {
  const int per = kRow / (dtype == TREE_BF16 ? 2 : 4);
  return (C + per - 1) / per;
}

struct ScanLayout {
  size_t link, end, kid, sib, info, edge, ctl, maps, dnode, carry, total;
};

ScanLayout scan_layout(const tree_plan_t* p, int C) {
  ScanLayout L{};
  const size_t tok = align256((size_t)p->n_tokens * 4), tiles = (size_t)scan_tiles(p);
  size_t o = 0;
  L.link = o;  o += tok;
  L.end = o;   o += tok;
  L.kid = o;   o += tok;
  L.sib = o;   o += tok;
  L.info = o;  o = align256(o + tiles * 4);
  L.edge = o;  o = align256(o + tiles * 4);
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
  return ScanWork{i32(L.link), i32(L.end), i32(L.kid), i32(L.sib), i32(L.info), i32(L.edge), i32(L.ctl),
                  f32(L.maps), f32(L.dnode), f32(L.carry)};
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

int scan_args(const tree_plan_t* plan, const int32_t* parent, const int32_t* node_len, int C, int dtype, int kind) {
  int rc = plan_ok(plan);
  if (rc) return rc;
  if (!plan->tok_node || !plan->tok_start || !plan->sub_end || !parent || !node_len) return TREE_ERR_ARG;
  if (plan->n_nodes <= 0 || C <= 0 || C > kMostChannels || C % 8 != 0) return TREE_ERR_SHAPE;
  if ((dtype != TREE_BF16 && dtype != TREE_F32) || (kind != TREE_GATE_SIGMOID && kind != TREE_GATE_LOG))
    return TREE_ERR_SHAPE;
  return TREE_OK;
}

// A call's buffers.  An output overlaps nothing, but that a per-token output may be a per-token input as a whole:
// a tile's inputs are in shared memory before its outputs are written, and no other tile reads them.
struct Buffer {
  const void* p;
  size_t bytes;
  bool tokens;
};
bool buffers_ok(const Buffer* out, int n_out, const Buffer* in, int n_in) {
  auto meet = [](const Buffer& a, const Buffer& b) { return buffers_meet(a.p, a.bytes, b.p, b.bytes); };
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < i; ++j)
      if (meet(out[i], out[j])) return false;
    for (int j = 0; j < n_in; ++j)
      if (meet(out[i], in[j]) && !(out[i].tokens && in[j].tokens && out[i].p == in[j].p)) return false;
  }
  return true;
}

ScanTree scan_tree(const tree_plan_t* plan, const int32_t* parent, const int32_t* node_len) {
  return ScanTree{plan->tok_node, plan->tok_start, plan->sub_end, parent, node_len,
                  plan->n_tokens, plan->n_nodes,   scan_tiles(plan)};
}

// a tensor [N][C] in boxes of a tile's tokens by a slab's channels; what lies outside reads as zero
template <typename T>
int scan_map(CUtensorMap* m, const void* base, int C, int N) {
  constexpr int box = kRow / (int)sizeof(T);
  return sizeof(T) == 2 ? make_tmap_bf16_2d(m, base, C, N, box, kTile) : make_tmap_f32_2d(m, base, C, N, box, kTile);
}

// The SMs of the current device; the kernel's dynamic shared memory is announced there, once a device.
template <auto KERN, int SMEM>
int announce(int* sms = nullptr) {
  static std::atomic<int> sms_of[64];              // one array a kernel; 0: not announced yet
  int dev = 0, n = 0;
  int rc = record_cuda(cudaGetDevice(&dev));
  if (rc) return rc;
  if (dev < 64) n = sms_of[dev].load(std::memory_order_acquire);
  if (!n) {
    rc = record_cuda(cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM));
    if (!rc) rc = record_cuda(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev));
    if (rc) return rc;
    if (dev < 64) sms_of[dev].store(n, std::memory_order_release);
  }
  if (sms) *sms = n;
  return TREE_OK;
}
// a block an SM, or one for each unit of work
template <auto KERN, int SMEM>
int scan_grid(int64_t units, unsigned* blocks) {
  int sms = 0;
  const int rc = announce<KERN, SMEM>(&sms);
  if (!rc) *blocks = (unsigned)std::min<int64_t>(units, sms);
  return rc;
}

// 12 bytes a channel are marked empty for each tile: a block for 1024 channels, as far as a grid goes; and one for the links
template <bool FWD>
int run_prepare(const ScanTree& t, const ScanWork& w, int C, float* rows, float* between, cudaStream_t s) {
  const dim3 grid((unsigned)t.n_tiles, 1u + (unsigned)std::min((C + 1023) / 1024, 65534));
  k_scan_prepare<FWD><<<grid, kTile, 0, s>>>(t, w, C, rows, between);
  return record_cuda(cudaGetLastError());
}

// `span` tokens a block
template <typename T, int KIND>
int run_step(const ScanFwd<T>& a, const void* gate, const void* x, int span, cudaStream_t s) {
  const int rc = announce<&k_scan_step<T, KIND>, step_smem<T>(kStepMost)>();
  if (rc) return rc;
  const int n = std::min(span, a.t.N), warps = (n + kStepTokens - 1) / kStepTokens;
  const dim3 grid((unsigned)a.slabs, (unsigned)((a.t.N + span - 1) / span));
  k_scan_step<T, KIND><<<grid, 32 * warps, step_smem<T>(n), s>>>(static_cast<const T*>(gate),
                                                                 static_cast<const T*>(x), span, a);
  return record_cuda(cudaGetLastError());
}
template <typename T, int KIND>
int run_fwd(const ScanFwd<T>& a, const CUtensorMap& tg, const CUtensorMap& tx, cudaStream_t s) {
  unsigned blocks = 0;
  const int rc = scan_grid<&k_scan_fwd<T, KIND>, scan_smem(kSlots)>((int64_t)a.t.n_tiles * a.slabs, &blocks);
  if (rc) return rc;
  k_scan_fwd<T, KIND><<<blocks, kScanThreads, scan_smem(kSlots), s>>>(tg, tx, a);
  return record_cuda(cudaGetLastError());
}
template <typename T, int KIND>
int run_bwd(const ScanBwd<T>& a, const CUtensorMap& tg, const CUtensorMap& tx, const CUtensorMap& td, cudaStream_t s) {
  unsigned blocks = 0;
  const int rc = scan_grid<&k_scan_bwd<T, KIND>, scan_smem(kSlots)>((int64_t)a.t.n_tiles * a.slabs, &blocks);
  if (rc) return rc;
  k_scan_bwd<T, KIND><<<blocks, kScanThreads, scan_smem(kSlots), s>>>(tg, tx, td, a);
  return record_cuda(cudaGetLastError());
}

template <typename T>
int scan_fwd(const ScanTree& t, int paths, int longest, const ScanWork& w, const void* gate, const void* x, const float* init, int C, int dtype,
             int kind, void* y, float* states, int32_t* status, cudaStream_t s) {
  const int slabs = scan_slabs(C, dtype);
  const ScanFwd<T> a{init, static_cast<T*>(y), states, t, w, C, slabs, status, wait_limit_ns()};
  // Few tokens, or a step: every node is a sequence of its own (as many paths as nodes), on average of at most a token
  // and none longer than kStepLongest.
  const bool step = paths == t.n_nodes && t.N <= t.n_nodes && longest <= kStepLongest && t.N <= 65535 * kTile;
  if (step || t.N <= kStepMost) {
    const int span = step ? kTile : kStepMost;         // (more blocks where they can be)
    return kind == TREE_GATE_SIGMOID ? run_step<T, TREE_GATE_SIGMOID>(a, gate, x, span, s)
                                     : run_step<T, TREE_GATE_LOG>(a, gate, x, span, s);
  }
  CUtensorMap tg, tx;
  int rc = scan_map<T>(&tg, gate, C, t.N);
  if (!rc) rc = scan_map<T>(&tx, x, C, t.N);
  if (rc) return rc;
  rc = run_prepare<true>(t, w, C, states, states + (size_t)t.n_nodes * C, s);
  if (rc) return rc;                                 // (the next kernel trusts what this one left)
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
  rc = run_prepare<false>(t, w, C, d_init, w.carry, s);
  if (rc) return rc;
  const ScanBwd<T> a{init, states, d_final, static_cast<T*>(dgate), static_cast<T*>(dx), d_init, t, w, C, slabs, status,
                     wait_limit_ns()};
  return kind == TREE_GATE_SIGMOID ? run_bwd<T, TREE_GATE_SIGMOID>(a, tg, tx, td, s)
                                   : run_bwd<T, TREE_GATE_LOG>(a, tg, tx, td, s);
}

}  // namespace
}  // namespace ta

using namespace ta;

extern "C" {

int64_t tree_scan_rows(const tree_plan_t* plan) {
  if (!plan || plan->n_tokens <= 0 || plan->n_nodes <= 0) return 0;
  return (int64_t)plan->n_nodes + scan_tiles(plan);
}

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
  const size_t tokens = (size_t)plan->n_tokens * C * (dtype == TREE_BF16 ? 2 : 4), nodes = (size_t)plan->n_nodes * C * 4;
  const Buffer out[] = {{workspace, scan_layout(plan, C).total, false}, {y, tokens, true},
                        {states, (size_t)tree_scan_rows(plan) * C * 4, false}};
  const Buffer in[] = {{gate, tokens, true}, {x, tokens, true}, {init, nodes, false}};
  if (!buffers_ok(out, 3, in, 3)) return TREE_ERR_ARG;
  rc = check_device();
  if (rc) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const ScanTree t = scan_tree(plan, parent, node_len);
  const ScanWork w = scan_work(workspace, scan_layout(plan, C));
  return dtype == TREE_BF16
             ? scan_fwd<__nv_bfloat16>(t, plan->n_paths, plan->max_len, w, gate, x, init, C, dtype, gate_kind, y, states, status_dev, s)
             : scan_fwd<float>(t, plan->n_paths, plan->max_len, w, gate, x, init, C, dtype, gate_kind, y, states, status_dev, s);
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
  const size_t tokens = (size_t)plan->n_tokens * C * (dtype == TREE_BF16 ? 2 : 4), nodes = (size_t)plan->n_nodes * C * 4;
  const Buffer out[] = {{workspace, scan_layout(plan, C).total, false}, {dgate, tokens, true}, {dx, tokens, true},
                        {d_init, nodes, false}};
  const Buffer in[] = {{gate, tokens, true}, {x, tokens, true}, {dy, tokens, true}, {init, nodes, false},
                       {d_final, nodes, false}, {states, (size_t)tree_scan_rows(plan) * C * 4, false}};
  if (!buffers_ok(out, 4, in, 6)) return TREE_ERR_ARG;
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
