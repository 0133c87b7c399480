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

constexpr int kScanWarps = 8;               // compute warps; one more warp loads
constexpr int kScanThreads = 32 * (kScanWarps + 1);
constexpr int kWarpTokens = TILE / kScanWarps;
constexpr int kRowBytes = 128;              // a tile's row: 64 bf16 or 32 fp32 channels, a word a lane
constexpr int kBoxBytes = TILE * kRowBytes;
constexpr int kScanGroup = 16;              // at most this many maps are joined to a state

constexpr int kLinkChain = -1;             // the token before on the path is the one before in packed order
constexpr int kLinkRoot = -2;              // the token starts from its node's initial state
constexpr int kFromTile = 1 << 30;         // mark on a node id (below 2^30): it ends in the tile at hand

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
// info: per tile, the kInfo bits.  flags: per tile and slab, how far it is.  ctl: the counter that
// hands out tiles (64 bits), and a word that stops every wait once one has run out of time.
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
enum : int { kFlagMap = 1, kFlagState = 2, kFlagAll = 3 };   // map, state behind it, nodes' rows: published

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

// One block a tile: links and info, the tile's flags cleared; and the rows that no tile writes are
// zeroed: those of nodes without tokens, and with `inner` of nodes that do not start from nothing.
__global__ void __launch_bounds__(TILE) k_scan_prepare(ScanTree t, ScanWork w, int slabs, int C, int inner,
                                                       float* rows) {
  __shared__ int bits;
  const int k = blockIdx.x, j = k * TILE + threadIdx.x;
  if (threadIdx.x == 0) bits = 0;
  if (k == 0 && threadIdx.x < 4) w.ctl[threadIdx.x] = 0;
  for (int i = threadIdx.x; i < slabs; i += TILE) w.flags[(size_t)k * slabs + i] = 0;
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
  if (!rows) return;
  for (int v = k; v < t.n_nodes; v += gridDim.x) {
    if (t.node_len[v] > 0 && !(inner && scan_token_ancestor(v, t) >= 0)) continue;
    for (int c = threadIdx.x; c < C; c += TILE) rows[(size_t)v * C + c] = 0.f;
  }
}

// p and b of one token
template <int KIND>
DEVI void gate_of(float g, float x, float& p, float& b) {
  if (KIND == TREE_GATE_SIGMOID) {
    const float e = expf(-fabsf(g)), r = __frcp_rn(1.f + e);
    const float small = e * r;                       // the smaller of a and 1 - a
    p = g > 0.f ? -small : small;
    b = (g > 0.f ? small : r) * x;
  } else {
    const float q = g > 0.f ? 0.f : g;               // NaN stays NaN
    const float m = expm1f(q);
    p = m > -0.5f ? m : expf(q);
    if (m == 0.f) p = -0.f;
    b = x;
  }
}
DEVI bool near_one(float p) { return __float_as_int(p) < 0; }
DEVI float decay(float p) { return near_one(p) ? 1.f + p : p; }
DEVI float lack(float p) { return near_one(p) ? -p : 1.f - p; }
// a h + b
DEVI float scan_step(float p, float b, float h) { return fmaf(p, h, b) + (near_one(p) ? h : 0.f); }
// a h
DEVI float scan_mul(float p, float h) { return fmaf(p, h, near_one(p) ? h : 0.f); }
// b, from x and p
template <int KIND>
DEVI float input_of(float p, float x) { return KIND == TREE_GATE_SIGMOID ? lack(p) * x : x; }

template <int KIND>
DEVI void gate_grad(float g, float x, float p, float before, float lam, float& dg, float& dx) {
  if (KIND == TREE_GATE_SIGMOID) {
    dx = lam * lack(p);
    dg = dx * decay(p) * (before - x);
  } else {
    dx = lam;
    dg = g > 0.f ? 0.f : lam * decay(p) * before;
  }
}

// A lane's word of a row: two bf16 channels or one fp32 channel.
template <typename T>
struct Lane;
template <>
struct Lane<__nv_bfloat16> {
  static constexpr int CH = 2;
  static DEVI void unpack(uint32_t w, float (&v)[2]) { v[0] = bf16lo(w); v[1] = bf16hi(w); }
  static DEVI uint32_t pack(const float (&v)[2]) { return pack_bf16(v[0], v[1]); }
};
template <>
struct Lane<float> {
  static constexpr int CH = 1;
  static DEVI void unpack(uint32_t w, float (&v)[1]) { v[0] = __uint_as_float(w); }
  static DEVI uint32_t pack(const float (&v)[1]) { return __float_as_uint(v[0]); }
};
// fp32 values of a lane's channels, past L1 (another block may have written them)
DEVI void ld_state(const float* p, float (&v)[2]) { const float2 a = __ldcg(reinterpret_cast<const float2*>(p)); v[0] = a.x; v[1] = a.y; }
DEVI void ld_state(const float* p, float (&v)[1]) { v[0] = __ldcg(p); }
// the same where `want`, else zeros; loads of a run of calls are all in flight before the first is used
DEVI void ld_state_if(const float* p, bool want, float (&v)[2]) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %3, 0;\n\tmov.f32 %0, 0f00000000;\n\tmov.f32 %1, 0f00000000;\n\t"
               "@q ld.global.cg.v2.f32 {%0, %1}, [%2];\n\t}"
               : "=&f"(v[0]), "=&f"(v[1]) : "l"(p), "r"((uint32_t)want) : "memory");
}
DEVI void ld_state_if(const float* p, bool want, float (&v)[1]) {
  asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\tmov.f32 %0, 0f00000000;\n\t"
               "@q ld.global.cg.f32 %0, [%1];\n\t}"
               : "=&f"(v[0]) : "l"(p), "r"((uint32_t)want) : "memory");
}
DEVI void st_state(float* p, const float (&v)[2]) { __stcg(reinterpret_cast<float2*>(p), make_float2(v[0], v[1])); }
DEVI void st_state(float* p, const float (&v)[1]) { __stcg(p, v[0]); }
// a lane's maps (A, B per channel)
DEVI void ld_map(const float* p, float (&A)[2], float (&B)[2]) {
  const float4 a = __ldcg(reinterpret_cast<const float4*>(p));
  A[0] = a.x; B[0] = a.y; A[1] = a.z; B[1] = a.w;
}
DEVI void ld_map(const float* p, float (&A)[1], float (&B)[1]) { const float2 a = __ldcg(reinterpret_cast<const float2*>(p)); A[0] = a.x; B[0] = a.y; }
DEVI void st_map(float* p, const float (&A)[2], const float (&B)[2]) { __stcg(reinterpret_cast<float4*>(p), make_float4(A[0], B[0], A[1], B[1])); }
DEVI void st_map(float* p, const float (&A)[1], const float (&B)[1]) { __stcg(reinterpret_cast<float2*>(p), make_float2(A[0], B[0])); }

DEVI int ld_acquire(const int32_t* p) {
  int v;
  asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
DEVI void st_release(int32_t* p, int v) {
  asm volatile("st.release.gpu.global.s32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Wait until *flag is at least `want`.  The first wait of the grid that runs out of time stops all others.
DEVI bool wait_flag(const int32_t* flag, int want, const WaitCtl& wc, int32_t* stop) {
  if (ld_acquire(flag) >= want) return true;
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (ld_acquire(flag) >= want) return true;
    if ((it & 15u) == 0) {
      if (*wc.abort_flag || ld_acquire(stop)) return false;
      if (global_timer_ns() - t0 > wc.limit_ns) {
        if (wc.status) atomicExch(wc.status, TREE_ERR_TIMEOUT);
        st_release(stop, 1);
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

// Shared by both kernels: a ring of stages, each one tile's rows of ARRAYS tensors.
template <int STAGES>
struct ScanShared {
  uint64_t full[STAGES], empty[STAGES];
  int tile[STAGES], slab[STAGES], info[STAGES], dist[STAGES];
  int abort_flag;
  int reset[kScanWarps];
  alignas(16) float maps[kScanWarps][64][2];       // per warp and channel: A, B
  float back[kScanWarps][64];                      // backward: what the warp adds to the gradient
  float in[64];
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

// Join `dist` maps to the state (or gradient) behind tile b, in the order in which the recurrence
// passes them; tiles b, b + step, ...  One warp; v holds the result.  False if a wait gave up.
template <int CH>
DEVI bool join_maps(float (&v)[CH], int b, int step, int dist, const float* state, const ScanWork& w, int slabs, int slab,
                    int C, int ch, bool on, const WaitCtl& wc) {
  const int lane = threadIdx.x & 31;
  bool ok = true;
  if (lane <= dist)
    ok = wait_flag(w.flags + (size_t)(b + step * lane) * slabs + slab, lane == 0 ? kFlagState : kFlagMap, wc,
                   w.ctl + 2);
  if (!__all_sync(0xffffffffu, ok)) return false;
  if (on) {
    ld_state(state, v);
#pragma unroll 4
    for (int j = 1; j <= dist; ++j) {
      float A[CH], B[CH];
      ld_map(w.maps + ((size_t)(b + step * j) * C + ch) * 2, A, B);
#pragma unroll
      for (int c = 0; c < CH; ++c) v[c] = fmaf(A[c], v[c], B[c]);
    }
  }
  return true;
}

// the warp's writes so far, and those that a barrier ordered before them, become visible with the flag
DEVI void publish(int32_t* flag, int value) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    __threadfence();
    st_release(flag, value);
  }
}

constexpr int kScanBar = 1;                // the named barrier of the compute warps
DEVI void scan_sync() {
  __syncwarp();
  named_bar_sync(kScanBar, 32 * kScanWarps);
}
DEVI bool scan_agree(bool ok) {            // true where every thread's is
  __syncwarp();
  return named_bar_and(kScanBar, 32 * kScanWarps, ok);
}

// One tile of the forward, a warp 16 consecutive tokens of it.  PLAIN: no break, no node's end, all 128
// tokens there.  False if a wait gave up.
template <typename T, int KIND, bool PLAIN, int STAGES>
DEVI bool scan_tile_fwd(const ScanFwd<T>& a, ScanShared<STAGES>& sh, const uint8_t* stage, uint64_t* empty, int k,
                        int slab, int info, int dist, const WaitCtl& wc) {
  constexpr int CH = Lane<T>::CH;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = slab * (kRowBytes / (int)sizeof(T)) + lane * CH;      // the lane's first channel
  const bool on = ch < a.C;
  const int t0 = k * TILE + warp * kWarpTokens;
  const bool in = info & kInfoIn, serial = !PLAIN && (info & kInfoSerial);
  float p[kWarpTokens][CH], b[kWarpTokens][CH];
  {
    const uint8_t* gs = stage + (size_t)(warp * kWarpTokens) * a.row_bytes + lane * 4;
    const uint8_t* xs = gs + kBoxBytes;
#pragma unroll
    for (int i = 0; i < kWarpTokens; ++i) {
      float g[CH], x[CH];
      Lane<T>::unpack(on ? *reinterpret_cast<const uint32_t*>(gs + i * a.row_bytes) : 0u, g);
      Lane<T>::unpack(on ? *reinterpret_cast<const uint32_t*>(xs + i * a.row_bytes) : 0u, x);
#pragma unroll
      for (int c = 0; c < CH; ++c) gate_of<KIND>(g[c], x[c], p[i][c], b[i][c]);
    }
  }
  __syncwarp();
  if (lane == 0) mbar_arrive(empty);                 // the stage is in registers
  // Breaks: `from` per lane and token, the node or kind of start; a start from outside the tile is folded
  // into its token, whose own map is then the constant b.
  int from = kLinkChain, end = -1;
  uint32_t breaks = 0, ends = 0, reset = 0;
  if (!PLAIN) {
    const int t = t0 + lane;
    bool ok = true;
    if (lane < kWarpTokens && t < a.t.N) {
      from = a.w.link[t];
      end = a.w.end[t];
      if (from >= 0) {
        const int ts = (a.t.tok_start[from] + a.t.node_len[from] - 1) / TILE;
        if (ts != k) ok = wait_flag(a.w.flags + (size_t)ts * a.slabs + slab, kFlagAll, wc, a.w.ctl + 2);
        else from |= kFromTile;                      // a node of this tile: its state comes while the tile runs
      }
    }
    if (!scan_agree(ok)) return false;
    breaks = __ballot_sync(0xffffffffu, from != kLinkChain);
    ends = __ballot_sync(0xffffffffu, end >= 0);
    reset = breaks & ~__ballot_sync(0xffffffffu, from >= 0 && (from & kFromTile));
    if (t0 > a.t.N - kWarpTokens) {                  // behind the last token h stays
#pragma unroll
      for (int i = 0; i < kWarpTokens; ++i)
        if (t0 + i >= a.t.N) {
#pragma unroll
          for (int c = 0; c < CH; ++c) { p[i][c] = -0.f; b[i][c] = 0.f; }
        }
    }
    if (reset) {
      float s[kWarpTokens][CH];
#pragma unroll
      for (int i = 0; i < kWarpTokens; ++i) {        // all loads first: none waits for another
        const int f = __shfl_sync(0xffffffffu, from, i);
        const float* row = f >= 0 ? a.states + (size_t)(f & ~kFromTile) * a.C
                                  : (a.init && f == kLinkRoot ? a.init + (size_t)a.t.tok_node[t0 + i] * a.C : nullptr);
        ld_state_if(row + ch, on && row && ((reset >> i) & 1u), s[i]);
      }
#pragma unroll
      for (int i = 0; i < kWarpTokens; ++i)
        if ((reset >> i) & 1u) {
#pragma unroll
          for (int c = 0; c < CH; ++c) b[i][c] = scan_step(p[i][c], b[i][c], s[i][c]);
        }
    }
  }
  // The warp's 16 steps as one map; behind a reset it is a constant.
  float A[CH], B[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) { A[c] = 1.f; B[c] = 0.f; }
  if (!serial) {
#pragma unroll
    for (int i = 0; i < kWarpTokens; ++i) {
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        B[c] = (!PLAIN && ((reset >> i) & 1u)) ? b[i][c] : scan_step(p[i][c], b[i][c], B[c]);
        A[c] = scan_mul(p[i][c], A[c]);
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      sh.maps[warp][lane * CH + c][0] = A[c];
      sh.maps[warp][lane * CH + c][1] = B[c];
    }
    if (!PLAIN && lane == 0) sh.reset[warp] = reset != 0;
  }
  scan_sync();
  int32_t* flag = a.w.flags + (size_t)k * a.slabs + slab;
  float* after = a.states + (size_t)(a.t.n_nodes + k) * a.C + ch;       // the state behind the tile
  const int last_flag = (info & kInfoSource) ? kFlagState : kFlagAll;
  // The map of the warps before this one (warp 0: of all, for the tile).
  const int upto = warp == 0 ? kScanWarps : warp;
  bool fixed = false;
#pragma unroll
  for (int c = 0; c < CH; ++c) { A[c] = 1.f; B[c] = 0.f; }
  if (!serial)
    for (int q = 0; q < upto; ++q) {
      const bool r = !PLAIN && sh.reset[q];
      fixed |= r;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const float qa = sh.maps[q][lane * CH + c][0], qb = sh.maps[q][lane * CH + c][1];
        B[c] = r ? qb : fmaf(qa, B[c], qb);
        A[c] *= qa;
      }
    }
  bool ok = true;
  if (warp == 0) {
    if (is_map_fwd(info) && (k + 1) % kScanGroup != 0 && k + 1 < a.tiles) {
      if (on) st_map(a.w.maps + ((size_t)k * a.C + ch) * 2, A, B);
      publish(flag, kFlagMap);
    }
    float h[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) h[c] = 0.f;
    if (in) {
      const int base = k - 1 - dist;
      ok = join_maps(h, base, 1, dist, a.states + (size_t)(a.t.n_nodes + base) * a.C + ch, a.w, a.slabs, slab, a.C, ch,
                     on, wc);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) sh.in[lane * CH + c] = h[c];
    if (!serial && ok) {
#pragma unroll
      for (int c = 0; c < CH; ++c) h[c] = fixed ? B[c] : fmaf(A[c], h[c], B[c]);
      if (on) st_state(after, h);
      publish(flag, last_flag);
    }
    fixed = false;
#pragma unroll
    for (int c = 0; c < CH; ++c) { A[c] = 1.f; B[c] = 0.f; }
  }
  if (!scan_agree(ok)) return false;
  // Now every h.
  float h[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    h[c] = sh.in[lane * CH + c];
    h[c] = fixed ? B[c] : (warp == 0 ? h[c] : fmaf(A[c], h[c], B[c]));
  }
  for (int turn = 0; turn < (serial ? kScanWarps : 1); ++turn) {
    if (!serial || turn == warp) {
      if (serial && warp > 0) {
#pragma unroll
        for (int c = 0; c < CH; ++c) h[c] = sh.in[lane * CH + c];
      }
      T* y = a.y + (size_t)t0 * a.C + ch;
#pragma unroll
      for (int i = 0; i < kWarpTokens; ++i) {
        if (!PLAIN && ((breaks >> i) & 1u) && !((reset >> i) & 1u)) {
          const int f = __shfl_sync(0xffffffffu, from, i) & ~kFromTile;
          if (on) ld_state(a.states + (size_t)f * a.C + ch, h);
        }
#pragma unroll
        for (int c = 0; c < CH; ++c)
          h[c] = (!PLAIN && ((reset >> i) & 1u)) ? b[i][c] : scan_step(p[i][c], b[i][c], h[c]);
        if (on && (PLAIN || t0 + i < a.t.N)) *reinterpret_cast<uint32_t*>(y + (size_t)i * a.C) = Lane<T>::pack(h);
        if (!PLAIN && ((ends >> i) & 1u)) {
          const int e = __shfl_sync(0xffffffffu, end, i);
          if (on) st_state(a.states + (size_t)e * a.C + ch, h);
        }
      }
      if (serial) {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < CH; ++c) sh.in[lane * CH + c] = h[c];
        if (warp == kScanWarps - 1 && on) st_state(after, h);
      }
    }
    if (serial) scan_sync();
  }
  if (!PLAIN && (serial || (info & kInfoSource))) {
    if (!serial) scan_sync();
    if (warp == 0) publish(flag, kFlagAll);
  }
  return true;
}

// One tile of the backward.  h is computed again from the state behind the tile before; the gradient runs
// from the last token to the first.  PLAIN: no break, nothing joins at a node's end, all 128 tokens there.
template <typename T, int KIND, bool PLAIN, int STAGES>
DEVI bool scan_tile_bwd(const ScanBwd<T>& a, ScanShared<STAGES>& sh, const uint8_t* stage, int k, int slab, int info,
                        int dist, const WaitCtl& wc) {
  constexpr int CH = Lane<T>::CH;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ch = slab * (kRowBytes / (int)sizeof(T)) + lane * CH;
  const bool on = ch < a.C;
  const int t0 = k * TILE + warp * kWarpTokens;
  const bool serial = !PLAIN && (info & kInfoSerialBack);
  const uint8_t* gs = stage + (size_t)(warp * kWarpTokens) * a.row_bytes + lane * 4;
  const uint8_t *xs = gs + kBoxBytes, *ds = xs + kBoxBytes;
  auto word = [&](const uint8_t* q, int i, float(&v)[CH]) {
    Lane<T>::unpack(on ? *reinterpret_cast<const uint32_t*>(q + i * a.row_bytes) : 0u, v);
  };
  float hin[CH];                                     // the state before the tile
  ld_state_if(a.states + (size_t)(a.t.n_nodes + k - 1) * a.C + ch, on && (info & kInfoIn), hin);
  float p[kWarpTokens][CH], before[kWarpTokens][CH];
  int from = kLinkChain, end = -1, kid = -1, sib = -1, own = -1;
  uint32_t breaks = 0, ends = 0;
  if (!PLAIN) {
    const int t = t0 + lane;
    bool ok = true;
    if (lane < kWarpTokens && t < a.t.N) {
      from = a.w.link[t];
      end = a.w.end[t];
      kid = a.w.kid[t];
      sib = a.w.sib[t];
      own = a.t.tok_node[t];
      if (kid >= 0) {
        const int tk = a.t.tok_start[kid] / TILE;
        if (tk != k) ok = wait_flag(a.w.flags + (size_t)tk * a.slabs + slab, kFlagAll, wc, a.w.ctl + 2);
      }
      if (ok && sib >= 0) {
        const int tk = a.t.tok_start[sib] / TILE;
        if (tk != k) ok = wait_flag(a.w.flags + (size_t)tk * a.slabs + slab, kFlagAll, wc, a.w.ctl + 2);
      }
    }
    if (!scan_agree(ok)) return false;
    breaks = __ballot_sync(0xffffffffu, from != kLinkChain);
    ends = __ballot_sync(0xffffffffu, kid >= 0 || (end >= 0 && a.d_final));
    if (breaks) {
#pragma unroll
      for (int i = 0; i < kWarpTokens; ++i) {        // where a break's h comes from
        const int f = __shfl_sync(0xffffffffu, from, i), v = __shfl_sync(0xffffffffu, own, i);
        const float* row = f >= 0 ? a.states + (size_t)f * a.C
                                  : (a.init && f == kLinkRoot ? a.init + (size_t)v * a.C : nullptr);
        ld_state_if(row + ch, on && row && ((breaks >> i) & 1u), before[i]);
      }
    }
  }
  // what joins the gradient at token i besides dy and the token behind it
  auto joins = [&](int i, float(&v)[CH]) {
    const int kd = __shfl_sync(0xffffffffu, kid, i), e = __shfl_sync(0xffffffffu, end, i);
    float r[CH];
    if (a.d_final) {
      ld_state_if(a.d_final + (size_t)e * a.C + ch, on, r);
#pragma unroll
      for (int c = 0; c < CH; ++c) v[c] += r[c];
    }
    ld_state_if(a.w.dnode + (size_t)kd * a.C + ch, on && kd >= 0, r);
#pragma unroll
    for (int c = 0; c < CH; ++c) v[c] += r[c];
  };
  // The warp's 16 steps as one map of h, and as one of the gradient (with the same factor).
  float A[CH], B[CH], R[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) { A[c] = 1.f; B[c] = 0.f; R[c] = 0.f; }
#pragma unroll
  for (int i = 0; i < kWarpTokens; ++i) {
    float g[CH], x[CH];
    word(gs, i, g);
    word(xs, i, x);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      float b;
      gate_of<KIND>(g[c], x[c], p[i][c], b);
      B[c] = scan_step(p[i][c], b, (!PLAIN && ((breaks >> i) & 1u)) ? before[i][c] : B[c]);
      A[c] = scan_mul(p[i][c], A[c]);
    }
  }
  if (!serial) {
#pragma unroll
    for (int i = kWarpTokens - 1; i >= 0; --i) {
      float d[CH];
      word(ds, i, d);
      if (!PLAIN && ((ends >> i) & 1u)) joins(i, d);
#pragma unroll
      for (int c = 0; c < CH; ++c)
        R[c] = (!PLAIN && ((breaks >> i) & 1u)) ? 0.f : scan_mul(p[i][c], d[c] + R[c]);
    }
  }
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    sh.maps[warp][lane * CH + c][0] = A[c];
    sh.maps[warp][lane * CH + c][1] = B[c];
    sh.back[warp][lane * CH + c] = R[c];
  }
  if (!PLAIN && lane == 0) sh.reset[warp] = breaks != 0;
  scan_sync();
  // h before the warp's tokens, then before each of them
  {
    float h[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) h[c] = hin[c];
    for (int q = 0; q < warp; ++q) {
      const bool r = !PLAIN && sh.reset[q];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const float qb = sh.maps[q][lane * CH + c][1];
        h[c] = r ? qb : fmaf(sh.maps[q][lane * CH + c][0], h[c], qb);
      }
    }
#pragma unroll
    for (int i = 0; i < kWarpTokens; ++i) {
      float x[CH];
      word(xs, i, x);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (PLAIN || !((breaks >> i) & 1u)) before[i][c] = h[c];
        h[c] = scan_step(p[i][c], input_of<KIND>(p[i][c], x[c]), before[i][c]);
      }
    }
  }
  // the map of the warps behind this one
  bool fixed = false;
#pragma unroll
  for (int c = 0; c < CH; ++c) { A[c] = 1.f; R[c] = 0.f; }
  auto add_warp = [&](int q) {
    const bool r = !PLAIN && sh.reset[q];
    fixed |= r;
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const float qa = sh.maps[q][lane * CH + c][0], qr = sh.back[q][lane * CH + c];
      R[c] = r ? qr : fmaf(qa, R[c], qr);
      A[c] *= qa;
    }
  };
  int32_t* flag = a.w.flags + (size_t)k * a.slabs + slab;
  bool ok = true;
  if (!serial)
    for (int q = kScanWarps - 1; q > warp; --q) add_warp(q);
  if (warp == 0) {
    const bool fixed1 = fixed;
    float A1[CH], R1[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) { A1[c] = A[c]; R1[c] = R[c]; }
    if (!serial) add_warp(0);
    if (is_map_bwd(info) && k % kScanGroup != 0) {
      if (on) st_map(a.w.maps + ((size_t)k * a.C + ch) * 2, A, R);
      publish(flag, kFlagMap);
    }
    float u[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) u[c] = 0.f;
    if (info & kInfoOut) {
      const int base = k + 1 + dist;
      ok = join_maps(u, base, -1, dist, a.w.carry + (size_t)base * a.C + ch, a.w, a.slabs, slab, a.C, ch, on, wc);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) sh.in[lane * CH + c] = u[c];
    if (!serial && ok) {
#pragma unroll
      for (int c = 0; c < CH; ++c) u[c] = fixed ? R[c] : fmaf(A[c], u[c], R[c]);
      if (on) st_state(a.w.carry + (size_t)k * a.C + ch, u);
      publish(flag, (info & kInfoBreak) ? kFlagState : kFlagAll);
    }
    fixed = fixed1;
#pragma unroll
    for (int c = 0; c < CH; ++c) { A[c] = A1[c]; R[c] = R1[c]; }
  }
  if (!scan_agree(ok)) return false;
  float u[CH];
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    u[c] = sh.in[lane * CH + c];
    if (warp != kScanWarps - 1) u[c] = fixed ? R[c] : fmaf(A[c], u[c], R[c]);
  }
  for (int turn = 0; turn < (serial ? kScanWarps : 1); ++turn) {
    if (!serial || turn == kScanWarps - 1 - warp) {
      if (serial) {
#pragma unroll
        for (int c = 0; c < CH; ++c) u[c] = sh.in[lane * CH + c];
      }
#pragma unroll
      for (int i = kWarpTokens - 1; i >= 0; --i) {
        float lam[CH], x[CH], g[CH], dg[CH], dx[CH];
        word(ds, i, lam);
        word(xs, i, x);
        if (KIND == TREE_GATE_LOG) word(gs, i, g);
        if (!PLAIN && ((ends >> i) & 1u)) joins(i, lam);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          lam[c] += u[c];
          gate_grad<KIND>(g[c], x[c], p[i][c], before[i][c], lam[c], dg[c], dx[c]);
          u[c] = scan_mul(p[i][c], lam[c]);
        }
        if (on && (PLAIN || t0 + i < a.t.N)) {
          const size_t at = (size_t)(t0 + i) * a.C + ch;
          *reinterpret_cast<uint32_t*>(a.dgate + at) = Lane<T>::pack(dg);
          *reinterpret_cast<uint32_t*>(a.dx + at) = Lane<T>::pack(dx);
        }
        if (!PLAIN && ((breaks >> i) & 1u)) {        // what this path hands to the state it started from
          const int f = __shfl_sync(0xffffffffu, from, i), v = __shfl_sync(0xffffffffu, own, i);
          const int sb = __shfl_sync(0xffffffffu, sib, i);
          float r[CH];
          ld_state_if(a.w.dnode + (size_t)sb * a.C + ch, on && sb >= 0, r);
#pragma unroll
          for (int c = 0; c < CH; ++c) r[c] += u[c];
          if (on && f >= 0) st_state(a.w.dnode + (size_t)v * a.C + ch, r);
          if (on && f == kLinkRoot && a.d_init) st_state(a.d_init + (size_t)v * a.C + ch, u);
#pragma unroll
          for (int c = 0; c < CH; ++c) u[c] = 0.f;
        }
      }
      if (serial) {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < CH; ++c) sh.in[lane * CH + c] = u[c];
        if (warp == 0 && on) st_state(a.w.carry + (size_t)k * a.C + ch, u);
      }
    }
    if (serial) scan_sync();
  }
  if (!PLAIN && (serial || (info & kInfoBreak))) {
    if (!serial) scan_sync();
    if (warp == 0) publish(flag, kFlagAll);
  }
  return true;
}

constexpr int kFwdStages = 3, kBwdStages = 2;      // 96 KB of copies a block, two blocks an SM
constexpr int scan_smem(int stages, int arrays) { return stages * arrays * kBoxBytes + 1024; }

DEVI uint8_t* scan_align(uint8_t* p) { return p + ((1024u - (smem_u32(p) & 1023u)) & 1023u); }

template <int STAGES>
DEVI void scan_init(ScanShared<STAGES>& sh) {
  if (threadIdx.x == 0) {
    sh.abort_flag = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&sh.full[s], 2);                   // the copies' announcement, and what tile it is
      mbar_init(&sh.empty[s], kScanWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
}

template <typename T, int KIND>
__global__ void __launch_bounds__(kScanThreads, 2) k_scan_fwd(const __grid_constant__ CUtensorMap tm_gate,
                                                              const __grid_constant__ CUtensorMap tm_x,
                                                              const ScanFwd<T> a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ ScanShared<kFwdStages> sh;
  uint8_t* stages = scan_align(smem_raw);
  scan_init(sh);
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  if (threadIdx.x >= 32 * kScanWarps) {
    const CUtensorMap* tm[2] = {&tm_gate, &tm_x};
    scan_loader<true>(sh, stages, tm, a.w, a.tiles, a.slabs, kRowBytes / (int)sizeof(T), TILE * a.row_bytes, wc);
    return;
  }
  for (int i = 0;; ++i) {
    const int s = i % kFwdStages;
    bool ok = scan_agree(mbar_wait(&sh.full[s], (i / kFwdStages) & 1, wc));
    if (!ok) break;
    const int k = sh.tile[s], slab = sh.slab[s], info = sh.info[s], dist = sh.dist[s];
    if (k < 0) break;
    const uint8_t* stage = stages + (size_t)s * 2 * kBoxBytes;
    if (!(info & (kInfoBreak | kInfoEnd)) && (k + 1) * (int64_t)TILE <= a.t.N)
      ok = scan_tile_fwd<T, KIND, true>(a, sh, stage, &sh.empty[s], k, slab, info, dist, wc);
    else
      ok = scan_tile_fwd<T, KIND, false>(a, sh, stage, &sh.empty[s], k, slab, info, dist, wc);
    if (!ok) {
      sh.abort_flag = 1;                           // the loading warp stops too
      break;
    }
  }
}

template <typename T, int KIND>
__global__ void __launch_bounds__(kScanThreads, 2) k_scan_bwd(const __grid_constant__ CUtensorMap tm_gate,
                                                              const __grid_constant__ CUtensorMap tm_x,
                                                              const __grid_constant__ CUtensorMap tm_dy,
                                                              const ScanBwd<T> a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ ScanShared<kBwdStages> sh;
  uint8_t* stages = scan_align(smem_raw);
  scan_init(sh);
  const WaitCtl wc{&sh.abort_flag, a.status, a.limit_ns};
  if (threadIdx.x >= 32 * kScanWarps) {
    const CUtensorMap* tm[3] = {&tm_gate, &tm_x, &tm_dy};
    scan_loader<false>(sh, stages, tm, a.w, a.tiles, a.slabs, kRowBytes / (int)sizeof(T), TILE * a.row_bytes, wc);
    return;
  }
  for (int i = 0;; ++i) {
    const int s = i % kBwdStages;
    bool ok = scan_agree(mbar_wait(&sh.full[s], (i / kBwdStages) & 1, wc));
    if (!ok) break;
    const int k = sh.tile[s], slab = sh.slab[s], info = sh.info[s], dist = sh.dist[s];
    if (k < 0) break;
    const uint8_t* stage = stages + (size_t)s * 3 * kBoxBytes;
    const bool plain = !(info & (kInfoBreak | kInfoSource)) && !((info & kInfoEnd) && a.d_final) &&
                       (k + 1) * (int64_t)TILE <= a.t.N;
    if (plain) ok = scan_tile_bwd<T, KIND, true>(a, sh, stage, k, slab, info, dist, wc);
    else ok = scan_tile_bwd<T, KIND, false>(a, sh, stage, k, slab, info, dist, wc);
    if (!ok) {
      sh.abort_flag = 1;
      break;
    }
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.empty[s]);
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
  if (plan->n_nodes <= 0 || plan->n_nodes >= kFromTile || C <= 0 || C % 8 != 0) return TREE_ERR_SHAPE;
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
  k_scan_prepare<<<(unsigned)t.n_tiles, TILE, 0, s>>>(t, w, slabs, C, 0, states);
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
  k_scan_prepare<<<(unsigned)t.n_tiles, TILE, 0, s>>>(t, w, slabs, C, 1, d_init);
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
