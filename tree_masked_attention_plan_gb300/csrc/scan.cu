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

#include "common.cuh"

namespace ta {
int make_tmap_bf16_2d(CUtensorMap* m, const void* base, int inner, int rows, int box_inner, int box_rows);  // host.cu

namespace {

constexpr int kScanWarps = 8;               // compute warps; one more warp loads, one joins
constexpr int kScanThreads = 32 * (kScanWarps + 2);
constexpr int kWarpTokens = TILE / kScanWarps;
constexpr int kRowBytes = 128;              // a tile's row: 64 bf16 or 32 fp32 channels, a word a lane
constexpr int kBoxBytes = TILE * kRowBytes;
constexpr int kScanGroup = 16;              // at most this many maps are joined to a state

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
};
// Maps and the states between tiles carry their own arrival: their rows hold this pattern, a NaN that no
// arithmetic gives, until they are written, and whoever needs one polls the value itself.  No flag and no
// fence stands between a tile and the next.
constexpr uint32_t kEmpty = 0xffffffffu;

// the tile is a plain map of the state before it / of the gradient behind it
DEVI bool is_map_fwd(int info) { return !(info & kInfoBreak); }
DEVI bool is_map_bwd(int info) { return !(info & (kInfoBreak | kInfoSource)) && (info & kInfoOut); }

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
DEVI Vec<CH> operator-(Vec<CH> a) {
#pragma unroll
  for (int c = 0; c < CH; ++c) a.v[c] = -a.v[c];
  return a;
}
template <int CH>
DEVI Vec<CH> operator-(Vec<CH> a, Vec<CH> b) { return a + (-b); }

// A decay a as p: -(1 - a) with the sign bit set where a >= 1/2, a itself elsewhere.
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
    for (int c = 0; c < CH; ++c)
      p.v[c] = n.v[c] <= -0.6931471805599453f ? e.v[c] : __uint_as_float(__float_as_uint(s.v[c]) | 0x80000000u);
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

template <typename T>
struct ScanFwd {
  const float* init;
  T* y;
  float* states;
  ScanTree t;
  ScanWork w;
  int C, slabs, tiles, row_bytes;
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
  int C, slabs, tiles, row_bytes;
  int32_t* status;
  uint64_t limit_ns;
};

// Shared by both kernels: a ring of stages, each one tile's rows of the staged tensors, and what the warps
// of a block tell each other, twice over: a warp may be a tile ahead of another.
template <int STAGES>
struct ScanShared {
  uint64_t full[STAGES], empty[STAGES], ready[2];  // ready: the state before (gradient behind) the tile is in `in`
  int tile[STAGES], slab[STAGES], info[STAGES], dist[STAGES];
  int abort_flag;
  int in_ok[2], reset[2][kScanWarps];
  alignas(16) float A[2][kScanWarps][64];          // per warp and channel: the map of its 16 tokens
  alignas(16) float B[2][kScanWarps][64];
  alignas(16) float R[2][kScanWarps][64];          // backward: that of the gradient is u -> A u + R
  alignas(16) float in[2][64];
  alignas(16) float carry[kScanWarps][64];         // behind (before) a warp, in tiles that go warp by warp
};

// The loading warp: takes tiles from the counter, starts their copies, and finds how many maps lie
// between the tile and the state it starts from.  FWD: that is the state behind the nearest tile before
// it that is no plain map or ends a group of kScanGroup; backward the same from the other side.
// Groups bound the maps that a tile joins; within one, no tile waits for a state to be handed on.
template <bool FWD, int STAGES, int ARRAYS>
DEVI void scan_loader(ScanShared<STAGES>& sh, uint8_t* stages, const CUtensorMap* const (&tm)[ARRAYS], const ScanWork& w,
                      int tiles, int slabs, int slab_ch, int box_bytes, const WaitCtl& wc) {
  const int lane = threadIdx.x & 31;
  int i = 0;
  bool live = true;
  for (; live; ++i) {
    const int s = i % STAGES;
    bool ok = true;
    // The second ticket waits for the first one's copies: all blocks have their first by then.  A block that
    // took two neighbouring tiles at once would keep the second's map back while others wait for it.
    if (lane == 0 && i == 1) ok = mbar_wait(&sh.full[0], 0, wc);
    if (lane == 0 && i >= STAGES) ok = mbar_wait(&sh.empty[s], ((i / STAGES) - 1) & 1, wc);
    if (!__all_sync(0xffffffffu, ok)) break;
    unsigned long long ticket = 0;
    if (lane == 0) ticket = atomicAdd(reinterpret_cast<unsigned long long*>(w.ctl), 1ull);
    ticket = __shfl_sync(0xffffffffu, ticket, 0);
    const unsigned long long turn = ticket / (unsigned)slabs;    // tile by tile, its slabs side by side
    live = turn < (unsigned)tiles;
    if (!live) {
      if (lane == 0) {
        sh.tile[s] = -1;
        mbar_arrive(&sh.full[s]);
        mbar_arrive(&sh.full[s]);
      }
      break;
    }
    const int slab = static_cast<int>(ticket - turn * (unsigned)slabs);
    const int k = FWD ? static_cast<int>(turn) : tiles - 1 - static_cast<int>(turn);
    if (lane == 0) {
      mbar_expect_tx(&sh.full[s], ARRAYS * box_bytes);
#pragma unroll
      for (int a = 0; a < ARRAYS; ++a)
        tma_load_2d(stages + (size_t)(s * ARRAYS + a) * kBoxBytes, tm[a], &sh.full[s], slab * slab_ch, k * TILE);
    }
    const int j = FWD ? k - lane : k + lane;
    const int info = (lane <= kScanGroup && j >= 0 && j < tiles) ? w.info[j] : kInfoBreak;
    const bool map = FWD ? is_map_fwd(info) && (j + 1) % kScanGroup != 0 : is_map_bwd(info) && j % kScanGroup != 0;
    const uint32_t run = __ballot_sync(0xffffffffu, map) >> 1;
    if (lane == 0) {
      sh.tile[s] = k;
      sh.slab[s] = slab;
      sh.info[s] = info;
      sh.dist[s] = __ffs(~run) - 1;
      mbar_arrive(&sh.full[s]);
    }
  }
  // every copy has landed before the block's shared memory goes, also where the compute warps gave up
  // (after the last ticket, stage i's earlier copy has been used, and its barrier is the end's)
  if (lane == 0)
    for (int q = max(0, i - STAGES + (live ? 0 : 1)); q < i; ++q) {
      const uint64_t t0 = global_timer_ns();
      while (!mbar_try_wait(&sh.full[q % STAGES], (q / STAGES) & 1) && global_timer_ns() - t0 < wc.limit_ns) {
      }
    }
}


constexpr int kBarMaps = 1;                // compute and joining warps: the tile's maps are in shared memory
constexpr int kBarTurn = 2;                // ... + warp: the warp before (behind) is done, in tiles that go warp by warp
constexpr int kBarDone = kBarTurn + kScanWarps;     // compute warps: the tile's rows are written
constexpr int kComputeThreads = 32 * kScanWarps, kMapThreads = kComputeThreads + 32;

DEVI void bar_sync(int id, int threads) {
  __syncwarp();
  named_bar_sync(id, threads);
}
DEVI void bar_arrive(int id, int threads) {
  __syncwarp();
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
DEVI bool bar_agree(int id, int threads, bool ok) {        // true where every thread's is
  __syncwarp();
  return named_bar_and(id, threads, ok);
}

// The warp's writes so far, and those that a barrier ordered before them, become visible with the flag.
DEVI void publish(int32_t* flag) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) set_release(flag, 1);
}

// The joining warp's part of a tile: the state before it (backward: the gradient behind it), from the state
// behind tile b and the maps of the `dist` tiles between, in the order in which the recurrence passes them;
// b, b + step, ... lead to the tile.  The maps are joined first, so that a state that arrives last is one
// step away from being handed on.
template <int CH>
struct Joiner {
  const ScanWork& w;
  int C, ch, b, step, dist;
  const float* state;                        // row of tile b, at the lane's channels
  bool on;
  static constexpr int BATCH = 5;
  DEVI const float* map(int j) const { return w.maps + ((size_t)(b + step * j) * C + ch) * 2; }
  // The joined state in v.  block: wait for what is missing; else false if anything is.
  DEVI bool join(Vec<CH>& v, bool block, const WaitCtl& wc) const {
    bool ok = true;
    Vec<CH> PA = vec<CH>(1.f), PB = vec<CH>(0.f);
    if (on) {
      for (int j0 = 1; j0 <= dist && ok; j0 += BATCH) {
        Vec<CH> A[BATCH], B[BATCH];
#pragma unroll
        for (int q = 0; q < BATCH; ++q)
          if (j0 + q <= dist) look_map(map(j0 + q), A[q], B[q]);
#pragma unroll
        for (int q = 0; q < BATCH; ++q) {
          if (j0 + q > dist) break;
          if (!(is_full(A[q]) && is_full(B[q])))
            ok = block && ok && wait_until([&] { look_map(map(j0 + q), A[q], B[q]); return is_full(A[q]) && is_full(B[q]); },
                                           wc, w.ctl + 2);
          PB = vfma(A[q], PB, B[q]);
          PA = PA * A[q];
        }
      }
      if (ok) {
        Vec<CH> u = look_state(state, v);
        if (!is_full(u))
          ok = block && wait_until([&] { u = look_state(state, u); return is_full(u); }, wc, w.ctl + 2);
        v = dist ? vfma(PA, u, PB) : u;
      }
    }
    return __all_sync(0xffffffffu, ok);
  }
};

// The joining warp's loop body, both directions: find the state before the tile (ahead of the compute
// warps where the tiles it needs are done), publish the tile's map and the state behind it.
// Returns false when the block has to stop.
template <bool FWD, int CH, int STAGES>
DEVI bool scan_join(ScanShared<STAGES>& sh, int i, const ScanWork& w, int C, int tiles, int slabs, float* rows, int slab_ch,
                    const WaitCtl& wc, bool& ok) {
  const int lane = threadIdx.x & 31, s = i % STAGES, buf = i & 1;
  ok = mbar_wait_warp(&sh.full[s], (i / STAGES) & 1, wc) && ok;
  int k = -1, slab = 0, info = 0, dist = 0;
  if (ok) { k = sh.tile[s]; slab = sh.slab[s]; info = sh.info[s]; dist = sh.dist[s]; }
  __syncwarp();
  if (lane == 0) mbar_arrive(&sh.empty[s]);
  const bool live = ok && k >= 0;
  const int ch = slab * slab_ch + lane * CH;
  const bool on = live && ch < C;
  const bool need = live && (info & (FWD ? kInfoIn : kInfoOut));
  const int b = FWD ? k - 1 - dist : k + 1 + dist;
  const Joiner<CH> j{w, C, ch, b, FWD ? 1 : -1, dist, rows + (size_t)(need ? b : 0) * C + ch, on};
  Vec<CH> v = vec<CH>(0.f);
  auto hand_in = [&](bool good) {
    sh_st<CH>(sh.in[buf], v);
    if (lane == 0) sh.in_ok[buf] = good;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.ready[buf]);
  };
  const bool joined = live && (!need || j.join(v, false, wc));
  if (joined) hand_in(true);
  if (!bar_agree(kBarMaps, kMapThreads, ok) || !live) return false;
  const bool serial = info & (FWD ? kInfoSerial : kInfoSerialBack);
  Vec<CH> A = vec<CH>(1.f), B = vec<CH>(0.f);
  bool fixed = false;
  if (!serial) {
#pragma unroll
    for (int n = 0; n < kScanWarps; ++n) {
      const int q = FWD ? n : kScanWarps - 1 - n;
      const bool r = sh.reset[buf][q];
      const Vec<CH> qa = sh_ld<CH>(sh.A[buf][q]), qb = sh_ld<CH>(FWD ? sh.B[buf][q] : sh.R[buf][q]);
      B = r ? qb : vfma(qa, B, qb);
      A = A * qa;
      fixed |= r;
    }
  }
  const bool map = FWD ? is_map_fwd(info) && (k + 1) % kScanGroup != 0 && k + 1 < tiles
                       : is_map_bwd(info) && k % kScanGroup != 0;
  if (map && on) hand_map(w.maps + ((size_t)k * C + ch) * 2, A, B);
  if (!joined) {
    ok = j.join(v, true, wc);
    hand_in(ok);
  }
  if (!serial && ok && on) hand_state(rows + (size_t)k * C + ch, fixed ? B : vfma(A, v, B));
  return true;                                 // a failed wait ends the block at the next agreement
}

// Forward, one tile, a warp 16 consecutive tokens of it.  First half: the maps to each token from the state
// before the warp, or from its last break.  PLAIN: no break, no node's end, all 128 tokens there.
template <int CH>
struct FwdTile {
  Vec<CH> A[kWarpTokens], B[kWarpTokens];
  int from, end;
  uint32_t breaks, ends, reset;              // a bit a token: breaks; ends; breaks that start outside the tile
};

template <typename T, int KIND, bool PLAIN, int STAGES, int CH>
DEVI bool fwd_first(FwdTile<CH>& f, const ScanFwd<T>& a, ScanShared<STAGES>& sh, const uint8_t* stage,
                    uint64_t* empty, int buf, int k, int slab, const WaitCtl& wc) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = slab * (kRowBytes / (int)sizeof(T)) + lane * CH;      // the lane's first channel
  const bool on = ch < a.C;
  const int t0 = k * TILE + warp * kWarpTokens;
  const uint8_t* gs = stage + (size_t)(warp * kWarpTokens) * a.row_bytes + (on ? lane * 4 : 0);
  const uint8_t* xs = gs + kBoxBytes;
  bool ok = true;
  if (!PLAIN) {
    f.from = kLinkChain;
    f.end = -1;
    bool tile = false;
    if (lane < kWarpTokens && t0 + lane < a.t.N) {
      f.from = a.w.link[t0 + lane];
      f.end = a.w.end[t0 + lane];
      if (f.from >= 0) {
        const int ts = (a.t.tok_start[f.from] + a.t.node_len[f.from] - 1) / TILE;
        tile = ts == k;
        if (!tile) ok = wait_rows(a.w.flags + (size_t)ts * a.slabs + slab, wc, a.w.ctl + 2);
      }
    }
    ok = __all_sync(0xffffffffu, ok);
    f.breaks = __ballot_sync(0xffffffffu, f.from != kLinkChain);
    f.ends = __ballot_sync(0xffffffffu, f.end >= 0);
    f.reset = f.breaks & ~__ballot_sync(0xffffffffu, tile);
    if (f.reset) {
#pragma unroll
      for (int i = 0; i < kWarpTokens; ++i) {        // what they start from: all loads first
        const int n = __shfl_sync(0xffffffffu, f.from, i);
        const float* row = n >= 0 ? a.states + (size_t)n * a.C
                                  : (a.init && n == kLinkRoot ? a.init + (size_t)a.t.tok_node[t0 + i] * a.C : nullptr);
        f.B[i] = ld_state_if(row + ch, on && row && ((f.reset >> i) & 1u), f.B[i]);
      }
    }
  }
  Vec<CH> A = vec<CH>(1.f), B = vec<CH>(0.f);
#pragma unroll
  for (int i = 0; i < kWarpTokens; ++i) {
    Vec<CH> p = gate_of<KIND>(Lane<T>::unpack(*reinterpret_cast<const uint32_t*>(gs + i * a.row_bytes)));
    Vec<CH> x = Lane<T>::unpack(*reinterpret_cast<const uint32_t*>(xs + i * a.row_bytes));
    if (!PLAIN) {
      if (t0 > a.t.N - 1 - i) {                      // behind the last token h stays
        p = vec<CH>(-0.f);
        x = vec<CH>(0.f);
      }
      if ((f.breaks >> i) & 1u) {
        A = vec<CH>(1.f);
        B = ((f.reset >> i) & 1u) ? f.B[i] : vec<CH>(0.f);
      }
    }
    B = advance<KIND>(p, x, B);
    A = decayed(p, A);
    f.A[i] = A;
    f.B[i] = B;
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(empty);                 // the stage is in registers
  sh_st(sh.A[buf][warp], A);
  sh_st(sh.B[buf][warp], B);
  if (lane == 0) sh.reset[buf][warp] = !PLAIN && f.reset != 0;
  return ok;
}

// Second half: the state before the warp, then every h.  Where breaks start from nodes that end in this
// very tile, the warps go one after the other.
template <typename T, bool PLAIN, int STAGES, int CH>
DEVI bool fwd_second(const FwdTile<CH>& f, const ScanFwd<T>& a, ScanShared<STAGES>& sh, int buf, uint32_t parity,
                     int k, int slab, int info, const WaitCtl& wc) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = slab * (kRowBytes / (int)sizeof(T)) + lane * CH;
  const bool on = ch < a.C, serial = !PLAIN && (info & kInfoSerial);
  const int t0 = k * TILE + warp * kWarpTokens;
  Vec<CH> A = vec<CH>(1.f), B = vec<CH>(0.f);
  bool fixed = false;
  if (!serial) {
#pragma unroll
    for (int q = 0; q < kScanWarps - 1; ++q) {
      if (q >= warp) break;
      const bool r = !PLAIN && sh.reset[buf][q];
      const Vec<CH> qa = sh_ld<CH>(sh.A[buf][q]), qb = sh_ld<CH>(sh.B[buf][q]);
      B = r ? qb : vfma(qa, B, qb);
      A = A * qa;
      fixed |= r;
    }
  }
  bool ok = mbar_wait_warp(&sh.ready[buf], parity, wc) && sh.in_ok[buf];
  Vec<CH> h = sh_ld<CH>(sh.in[buf]);                 // the state before the tile
  if (!serial) {
    if (warp > 0) h = fixed ? B : vfma(A, h, B);
  } else if (warp > 0) {
    bar_sync(kBarTurn + warp, 64);
    h = sh_ld<CH>(sh.carry[warp - 1]);
  }
  T* y = a.y + (size_t)t0 * a.C + ch;
  if (PLAIN) {
    if (on && ok) {
#pragma unroll
      for (int i = 0; i < kWarpTokens; ++i)
        *reinterpret_cast<uint32_t*>(y + (size_t)i * a.C) = Lane<T>::pack(vfma(f.A[i], h, f.B[i]));
    }
    return ok;
  }
  // Walk over the tokens: h the state that the run at hand started from, `set` where that is in B already.
  auto walk = [&](Vec<CH> h, bool write_y, bool write_ends) {
    bool set = false;
    Vec<CH> v = h;
#pragma unroll
    for (int i = 0; i < kWarpTokens; ++i) {
      if ((f.breaks >> i) & 1u) {
        set = (f.reset >> i) & 1u;
        if (!set) h = ld_state_if(a.states + (size_t)__shfl_sync(0xffffffffu, f.from, i) * a.C + ch, on, h);
      }
      v = set ? f.B[i] : vfma(f.A[i], h, f.B[i]);
      if (write_y && on && t0 + i < a.t.N) *reinterpret_cast<uint32_t*>(y + (size_t)i * a.C) = Lane<T>::pack(v);
      if (write_ends && ((f.ends >> i) & 1u)) {
        const int e = __shfl_sync(0xffffffffu, f.end, i);
        if (on) st_state(a.states + (size_t)e * a.C + ch, v);
      }
    }
    return v;
  };
  int32_t* flag = a.w.flags + (size_t)k * a.slabs + slab;
  if (!serial) {
    if (ok) walk(h, true, true);
    if (info & kInfoSource) {
      bar_sync(kBarDone, kComputeThreads);
      if (warp == 0 && ok) publish(flag);
    }
    return ok;
  }
  // what the next warps wait for first: ends and the state behind the warp
  const Vec<CH> v = ok ? walk(h, false, true) : h;
  if (warp < kScanWarps - 1) {
    sh_st(sh.carry[warp], v);
    bar_arrive(kBarTurn + warp + 1, 64);
  } else if (ok) {
    if (on) hand_state(a.states + (size_t)(a.t.n_nodes + k) * a.C + ch, v);
    publish(flag);
  }
  if (ok) walk(h, true, false);
  return ok;
}

// Backward, one tile.  First half: p of every token, and the warp's 16 steps as a map of h and as one of the
// gradient.  PLAIN: no break, nothing joins at a node's end, all 128 tokens there.
template <int CH>
struct BwdTile {
  Vec<CH> p[kWarpTokens], before[kWarpTokens];
  Vec<CH> hin;
  int from, end, kid, sib, own;
  uint32_t breaks, ends;
};

// A warp's rows of a stage: word i of the gate's, x's and dy's
template <typename T>
struct Rows {
  const uint8_t* base;
  int stride;
  template <int WHICH>
  DEVI Vec<Lane<T>::CH> at(int i) const {
    return Lane<T>::unpack(*reinterpret_cast<const uint32_t*>(base + WHICH * kBoxBytes + i * stride));
  }
};

// what joins the gradient at token i besides dy and the token behind it
template <typename T, int CH>
DEVI Vec<CH> joins_at(const BwdTile<CH>& f, const ScanBwd<T>& a, int i, int ch, bool on) {
  const int kd = __shfl_sync(0xffffffffu, f.kid, i), e = __shfl_sync(0xffffffffu, f.end, i);
  const Vec<CH> d = ld_state_if(a.d_final + (size_t)e * a.C + ch, on && a.d_final, Vec<CH>());
  return d + ld_state_if(a.w.dnode + (size_t)kd * a.C + ch, on && kd >= 0, Vec<CH>());
}

template <typename T, int KIND, bool PLAIN, int STAGES, int CH>
DEVI bool bwd_first(BwdTile<CH>& f, const ScanBwd<T>& a, ScanShared<STAGES>& sh, const Rows<T>& rows, int buf, int k,
                    int slab, int info, const WaitCtl& wc) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = slab * (kRowBytes / (int)sizeof(T)) + lane * CH;
  const bool on = ch < a.C, serial = !PLAIN && (info & kInfoSerialBack);
  const int t0 = k * TILE + warp * kWarpTokens;
  bool ok = true;
  f.hin = ld_state_if(a.states + (size_t)(a.t.n_nodes + k - 1) * a.C + ch, on && (info & kInfoIn), f.hin);
  f.breaks = f.ends = 0;
  if (!PLAIN) {
    f.from = kLinkChain;
    f.end = f.kid = f.sib = f.own = -1;
    if (lane < kWarpTokens && t0 + lane < a.t.N) {
      const int t = t0 + lane;
      f.from = a.w.link[t];
      f.end = a.w.end[t];
      f.kid = a.w.kid[t];
      f.sib = a.w.sib[t];
      f.own = a.t.tok_node[t];
      if (f.kid >= 0) {
        const int tk = a.t.tok_start[f.kid] / TILE;
        if (tk != k) ok = wait_rows(a.w.flags + (size_t)tk * a.slabs + slab, wc, a.w.ctl + 2);
      }
      if (ok && f.sib >= 0) {
        const int tk = a.t.tok_start[f.sib] / TILE;
        if (tk != k) ok = wait_rows(a.w.flags + (size_t)tk * a.slabs + slab, wc, a.w.ctl + 2);
      }
    }
    ok = __all_sync(0xffffffffu, ok);
    f.breaks = __ballot_sync(0xffffffffu, f.from != kLinkChain);
    f.ends = __ballot_sync(0xffffffffu, f.kid >= 0 || (f.end >= 0 && a.d_final));
    if (f.breaks) {
#pragma unroll
      for (int i = 0; i < kWarpTokens; ++i) {        // where a break's h comes from
        const int n = __shfl_sync(0xffffffffu, f.from, i), v = __shfl_sync(0xffffffffu, f.own, i);
        const float* row = n >= 0 ? a.states + (size_t)n * a.C
                                  : (a.init && n == kLinkRoot ? a.init + (size_t)v * a.C : nullptr);
        f.before[i] = ld_state_if(row + ch, on && row && ((f.breaks >> i) & 1u), f.before[i]);
      }
    }
  }
  Vec<CH> A = vec<CH>(1.f), B = vec<CH>(0.f), R = vec<CH>(0.f);
#pragma unroll
  for (int i = 0; i < kWarpTokens; ++i) {
    f.p[i] = gate_of<KIND>(rows.template at<0>(i));
    if (!PLAIN && ((f.breaks >> i) & 1u)) B = f.before[i];
    B = advance<KIND>(f.p[i], rows.template at<1>(i), B);
    A = decayed(f.p[i], A);
  }
  if (!serial) {
#pragma unroll
    for (int i = kWarpTokens - 1; i >= 0; --i) {
      Vec<CH> d = rows.template at<2>(i);
      if (!PLAIN && ((f.ends >> i) & 1u)) d = d + joins_at(f, a, i, ch, on);
      R = decayed(f.p[i], d + R);
      if (!PLAIN && ((f.breaks >> i) & 1u)) R = vec<CH>(0.f);
    }
  }
  sh_st(sh.A[buf][warp], A);
  sh_st(sh.B[buf][warp], B);
  sh_st(sh.R[buf][warp], R);
  if (lane == 0) sh.reset[buf][warp] = f.breaks != 0;
  return ok;
}

// Second half: h before every token, then the gradients from the last token to the first.
template <typename T, int KIND, bool PLAIN, int STAGES, int CH>
DEVI bool bwd_second(BwdTile<CH>& f, const ScanBwd<T>& a, ScanShared<STAGES>& sh, const Rows<T>& rows, int buf,
                     uint32_t parity, int k, int slab, int info, const WaitCtl& wc) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = slab * (kRowBytes / (int)sizeof(T)) + lane * CH;
  const bool on = ch < a.C, serial = !PLAIN && (info & kInfoSerialBack);
  const int t0 = k * TILE + warp * kWarpTokens;
  Vec<CH> h = f.hin;
#pragma unroll
  for (int q = 0; q < kScanWarps - 1; ++q) {
    if (q >= warp) break;
    const Vec<CH> qb = sh_ld<CH>(sh.B[buf][q]);
    h = (!PLAIN && sh.reset[buf][q]) ? qb : vfma(sh_ld<CH>(sh.A[buf][q]), h, qb);
  }
#pragma unroll
  for (int i = 0; i < kWarpTokens; ++i) {
    if (PLAIN || !((f.breaks >> i) & 1u)) f.before[i] = h;
    h = advance<KIND>(f.p[i], rows.template at<1>(i), f.before[i]);
  }
  Vec<CH> A = vec<CH>(1.f), R = vec<CH>(0.f);
  bool fixed = false;
  if (!serial) {
#pragma unroll
    for (int q = kScanWarps - 1; q > 0; --q) {
      if (q <= warp) break;
      const bool r = !PLAIN && sh.reset[buf][q];
      const Vec<CH> qa = sh_ld<CH>(sh.A[buf][q]), qr = sh_ld<CH>(sh.R[buf][q]);
      R = r ? qr : vfma(qa, R, qr);
      A = A * qa;
      fixed |= r;
    }
  }
  const bool ok = mbar_wait_warp(&sh.ready[buf], parity, wc) && sh.in_ok[buf];
  Vec<CH> u = sh_ld<CH>(sh.in[buf]);                 // the gradient behind the tile
  if (!serial) {
    if (warp < kScanWarps - 1) u = fixed ? R : vfma(A, u, R);
  } else if (warp < kScanWarps - 1) {
    bar_sync(kBarTurn + warp, 64);
    u = sh_ld<CH>(sh.carry[warp + 1]);
  }
  if (ok) {
#pragma unroll
    for (int i = kWarpTokens - 1; i >= 0; --i) {
      Vec<CH> lam = rows.template at<2>(i) + u;
      if (!PLAIN && ((f.ends >> i) & 1u)) lam = lam + joins_at(f, a, i, ch, on);
      const Vec<CH> p = f.p[i];
      u = decayed(p, lam);
      Vec<CH> dx, dg;
      if (KIND == TREE_GATE_SIGMOID) {
        Vec<CH> m, s;                                // the smaller of a and 1 - a; 1 - a
#pragma unroll
        for (int c = 0; c < CH; ++c) m.v[c] = fabsf(p.v[c]);
        s = pick(p, m, vec<CH>(1.f) - m);
        dx = lam * s;
        dg = lam * (vfma(-m, m, m) * (f.before[i] - rows.template at<1>(i)));
      } else {
        dx = lam;
        dg = u * f.before[i];
        const Vec<CH> g = rows.template at<0>(i);
#pragma unroll
        for (int c = 0; c < CH; ++c) dg.v[c] = g.v[c] > 0.f ? 0.f : dg.v[c];
      }
      if (on && (PLAIN || t0 + i < a.t.N)) {
        const size_t at = (size_t)(t0 + i) * a.C + ch;
        *reinterpret_cast<uint32_t*>(a.dgate + at) = Lane<T>::pack(dg);
        *reinterpret_cast<uint32_t*>(a.dx + at) = Lane<T>::pack(dx);
      }
      if (!PLAIN && ((f.breaks >> i) & 1u)) {        // what this path hands to the state it started from
        const int n = __shfl_sync(0xffffffffu, f.from, i), v = __shfl_sync(0xffffffffu, f.own, i);
        const int sb = __shfl_sync(0xffffffffu, f.sib, i);
        const Vec<CH> later = ld_state_if(a.w.dnode + (size_t)sb * a.C + ch, on && sb >= 0, u);
        if (on && n >= 0) st_state(a.w.dnode + (size_t)v * a.C + ch, u + later);
        if (on && n == kLinkRoot && a.d_init) st_state(a.d_init + (size_t)v * a.C + ch, u);
        u = vec<CH>(0.f);
      }
    }
  }
  if (PLAIN) return ok;
  int32_t* flag = a.w.flags + (size_t)k * a.slabs + slab;
  if (serial) {
    if (warp > 0) {
      sh_st(sh.carry[warp], u);
      bar_arrive(kBarTurn + warp - 1, 64);
    } else if (ok) {
      if (on) hand_state(a.w.carry + (size_t)k * a.C + ch, u);
      publish(flag);
    }
  } else if (info & kInfoBreak) {
    bar_sync(kBarDone, kComputeThreads);
    if (warp == 0 && ok) publish(flag);
  }
  return ok;
}

constexpr int kFwdStages = 2, kBwdStages = 2;
constexpr int scan_smem(int stages, int arrays) { return stages * arrays * kBoxBytes + 1024; }

DEVI uint8_t* scan_align(uint8_t* p) { return p + ((1024u - (smem_u32(p) & 1023u)) & 1023u); }

template <int STAGES>
DEVI void scan_init(ScanShared<STAGES>& sh) {
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sh.full[s], 2);                   // the copies' announcement, and what tile it is
      mbar_init(&sh.empty[s], kScanWarps + 1);     // the compute warps and the joining warp
    }
    mbar_init(&sh.ready[0], 1);
    mbar_init(&sh.ready[1], 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
}

// Warps 0-7 compute, 8 loads, 9 joins.  The three agree once a tile (kBarMaps) whether all goes well; after a
// wait that gave up they leave together there.
template <typename T, int KIND>
__global__ void __launch_bounds__(kScanThreads, 2) k_scan_fwd(const __grid_constant__ CUtensorMap tm_gate,
                                                              const __grid_constant__ CUtensorMap tm_x,
                                                              const ScanFwd<T> a) {
  constexpr int CH = Lane<T>::CH, SLAB = kRowBytes / (int)sizeof(T);
  extern __shared__ uint8_t smem_raw[];
  __shared__ ScanShared<kFwdStages> sh;
  uint8_t* stages = scan_align(smem_raw);
  scan_init(sh);
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  const int warp = threadIdx.x >> 5;
  if (warp == kScanWarps) {
    const CUtensorMap* tm[2] = {&tm_gate, &tm_x};
    scan_loader<true>(sh, stages, tm, a.w, a.tiles, a.slabs, SLAB, TILE * a.row_bytes, wc);
    return;
  }
  bool ok = true;
  if (warp == kScanWarps + 1) {
    for (int i = 0; scan_join<true, CH>(sh, i, a.w, a.C, a.tiles, a.slabs, a.states + (size_t)a.t.n_nodes * a.C, SLAB,
                                        wc, ok);
         ++i) {
    }
    return;
  }
  FwdTile<CH> f;
  for (int i = 0;; ++i) {
    const int s = i % kFwdStages, buf = i & 1;
    ok = mbar_wait_warp(&sh.full[s], (i / kFwdStages) & 1, wc) && ok;
    int k = -1, slab = 0, info = 0;
    if (ok) { k = sh.tile[s]; slab = sh.slab[s]; info = sh.info[s]; }
    const bool plain = !(info & (kInfoBreak | kInfoEnd)) && (k + 1) * (int64_t)TILE <= a.t.N;
    const uint8_t* stage = stages + (size_t)s * 2 * kBoxBytes;
    if (k >= 0)
      ok = plain ? fwd_first<T, KIND, true>(f, a, sh, stage, &sh.empty[s], buf, k, slab, wc)
                 : fwd_first<T, KIND, false>(f, a, sh, stage, &sh.empty[s], buf, k, slab, wc);
    if (!bar_agree(kBarMaps, kMapThreads, ok)) {
      sh.abort_flag = 1;                           // the loading warp stops too
      break;
    }
    if (k < 0) break;
    ok = plain ? fwd_second<T, true>(f, a, sh, buf, (i >> 1) & 1, k, slab, info, wc)
               : fwd_second<T, false>(f, a, sh, buf, (i >> 1) & 1, k, slab, info, wc);
  }
}

template <typename T, int KIND>
__global__ void __launch_bounds__(kScanThreads, 2) k_scan_bwd(const __grid_constant__ CUtensorMap tm_gate,
                                                              const __grid_constant__ CUtensorMap tm_x,
                                                              const __grid_constant__ CUtensorMap tm_dy,
                                                              const ScanBwd<T> a) {
  constexpr int CH = Lane<T>::CH, SLAB = kRowBytes / (int)sizeof(T);
  extern __shared__ uint8_t smem_raw[];
  __shared__ ScanShared<kBwdStages> sh;
  uint8_t* stages = scan_align(smem_raw);
  scan_init(sh);
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == kScanWarps) {
    const CUtensorMap* tm[3] = {&tm_gate, &tm_x, &tm_dy};
    scan_loader<false>(sh, stages, tm, a.w, a.tiles, a.slabs, SLAB, TILE * a.row_bytes, wc);
    return;
  }
  bool ok = true;
  if (warp == kScanWarps + 1) {
    for (int i = 0; scan_join<false, CH>(sh, i, a.w, a.C, a.tiles, a.slabs, a.w.carry, SLAB, wc, ok); ++i) {
    }
    return;
  }
  BwdTile<CH> f;
  for (int i = 0;; ++i) {
    const int s = i % kBwdStages, buf = i & 1;
    ok = mbar_wait_warp(&sh.full[s], (i / kBwdStages) & 1, wc) && ok;
    int k = -1, slab = 0, info = 0;
    if (ok) { k = sh.tile[s]; slab = sh.slab[s]; info = sh.info[s]; }
    const bool plain = !(info & (kInfoBreak | kInfoSource)) && !((info & kInfoEnd) && a.d_final) &&
                       (k + 1) * (int64_t)TILE <= a.t.N;
    const bool on = slab * SLAB + lane * CH < a.C;
    const Rows<T> rows{stages + (size_t)s * 3 * kBoxBytes + (size_t)(warp * kWarpTokens) * a.row_bytes +
                           (on ? lane * 4 : 0),
                       a.row_bytes};
    if (k >= 0)
      ok = plain ? bwd_first<T, KIND, true>(f, a, sh, rows, buf, k, slab, info, wc)
                 : bwd_first<T, KIND, false>(f, a, sh, rows, buf, k, slab, info, wc);
    if (!bar_agree(kBarMaps, kMapThreads, ok)) {
      sh.abort_flag = 1;
      break;
    }
    if (k < 0) break;
    ok = plain ? bwd_second<T, KIND, true>(f, a, sh, rows, buf, (i >> 1) & 1, k, slab, info, wc)
               : bwd_second<T, KIND, false>(f, a, sh, rows, buf, (i >> 1) & 1, k, slab, info, wc);
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.empty[s]);
  }
}

// ---------------------------------------------------------------------------------------------
// host side

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// slabs of 128 bytes of channels: counted for the narrower type, which has the more of them
int scan_slabs(int C, int dtype) {
  const int per = kRowBytes / (dtype == TREE_BF16 ? 2 : 4);
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

// a tensor [N][C] in boxes of 128 tokens by a slab's channels (all C where there are fewer)
template <typename T>
int scan_map(CUtensorMap* m, const void* base, int C, int N) {
  const int box = std::min(C, kRowBytes / (int)sizeof(T));
  return sizeof(T) == 2 ? make_tmap_bf16_2d(m, base, C, N, box, TILE) : make_tmap_f32_2d(m, base, C, N, box, TILE);
}

// as many blocks as run at once (two an SM), or one for each unit of work
template <typename Kern>
int scan_grid(Kern kern, int smem, int64_t units, unsigned* blocks) {
  int rc = record_cuda(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  int dev = 0, sms = 0;
  if (!rc) rc = record_cuda(cudaGetDevice(&dev));
  if (!rc) rc = record_cuda(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  *blocks = (unsigned)std::min<int64_t>(units, 2 * (int64_t)sms);
  return rc;
}

// 12 bytes a channel are marked empty for each tile: a block for 1024 channels
dim3 prepare_grid(const ScanTree& t, int C) { return dim3((unsigned)t.n_tiles, (unsigned)((C + 1023) / 1024)); }

template <typename T, int KIND>
int run_fwd(const ScanFwd<T>& a, const CUtensorMap& tg, const CUtensorMap& tx, cudaStream_t s) {
  constexpr int smem = scan_smem(kFwdStages, 2);
  unsigned blocks = 0;
  const int rc = scan_grid(k_scan_fwd<T, KIND>, smem, (int64_t)a.tiles * a.slabs, &blocks);
  if (rc) return rc;
  k_scan_fwd<T, KIND><<<blocks, kScanThreads, smem, s>>>(tg, tx, a);
  return record_cuda(cudaGetLastError());
}
template <typename T, int KIND>
int run_bwd(const ScanBwd<T>& a, const CUtensorMap& tg, const CUtensorMap& tx, const CUtensorMap& td, cudaStream_t s) {
  constexpr int smem = scan_smem(kBwdStages, 3);
  unsigned blocks = 0;
  const int rc = scan_grid(k_scan_bwd<T, KIND>, smem, (int64_t)a.tiles * a.slabs, &blocks);
  if (rc) return rc;
  k_scan_bwd<T, KIND><<<blocks, kScanThreads, smem, s>>>(tg, tx, td, a);
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
  const ScanFwd<T> a{init, static_cast<T*>(y), states, t, w, C, slabs, t.n_tiles,
                     std::min(C * (int)sizeof(T), kRowBytes), status, wait_limit_ns()};
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
  const ScanBwd<T> a{init, states, d_final, static_cast<T*>(dgate), static_cast<T*>(dx), d_init, t, w, C, slabs,
                     t.n_tiles, std::min(C * (int)sizeof(T), kRowBytes), status, wait_limit_ns()};
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
