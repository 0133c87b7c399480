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
// Precision: states, gates and gradients are fp32.  A decay close to one is held as what it
// lacks to one: p = -(1 - a) where a > 1/2, p = a elsewhere, so that a memory of thousands of
// tokens does not lose its length to the rounding of a; the step h + (p h + b) then adds a small
// increment to h.
#include <algorithm>

#include "common.cuh"

namespace ta {
namespace {

constexpr int kLinkChain = -1;             // the token before on the path is the one before in packed order
constexpr int kLinkRoot = -2;              // the token starts from its node's initial state

struct ScanTree {
  const int32_t* tok_node;
  const int32_t* tok_start;
  const int32_t* sub_end;
  const int32_t* parent;
  const int32_t* node_len;
  int N, n_nodes;
};

// Per packed token, in the workspace:
//   link  kLinkChain, kLinkRoot, or the node whose final state the token starts from (a break)
//   end   the token's node if it is the node's last token, else -1
//   kid   for a node's last token: the second of the nodes that start from it (the first one is its
//         successor in packed order), -1 if there is none
//   sib   for a break: the next node after its own that starts from the same state, -1 if none
struct ScanLinks {
  int32_t *link, *end, *kid, *sib;
};

DEVI int scan_token_ancestor(int v, const ScanTree& t) {
  int a = t.parent[v];
  for (int guard = 0; a >= 0 && a < t.n_nodes && t.node_len[a] == 0 && guard < t.n_nodes; ++guard) a = t.parent[a];
  return (a >= 0 && a < t.n_nodes && t.node_len[a] > 0) ? a : -1;
}

__global__ void __launch_bounds__(256) k_scan_links(ScanTree t, ScanLinks l) {
  const int j = blockIdx.x * blockDim.x + threadIdx.x;
  if (j >= t.N) return;
  const int v = t.tok_node[j];
  int link = kLinkChain, sib = -1, end = -1, kid = -1;
  if (j == t.tok_start[v]) {
    const int a = scan_token_ancestor(v, t);
    if (a < 0) {
      link = kLinkRoot;
    } else if (t.tok_start[a] + t.node_len[a] != j) {
      link = a;
      const int next = t.sub_end[v];
      if (next < t.sub_end[a]) sib = t.tok_node[next];
    }
  }
  if (j == t.tok_start[v] + t.node_len[v] - 1) {
    end = v;
    if (j + 1 < t.sub_end[v]) {
      const int next = t.sub_end[t.tok_node[j + 1]];
      if (next < t.sub_end[v]) kid = t.tok_node[next];
    }
  }
  l.link[j] = link;
  l.end[j] = end;
  l.kid[j] = kid;
  l.sib[j] = sib;
}

// rows of `rows` whose node holds no tokens, and the rows of nodes that do not start from nothing
// if `inner` is set, are zeroed
__global__ void __launch_bounds__(256) k_scan_zero_rows(ScanTree t, int C, int inner, float* rows) {
  for (int v = blockIdx.x; v < t.n_nodes; v += gridDim.x) {
    if (t.node_len[v] > 0 && !(inner && scan_token_ancestor(v, t) >= 0)) continue;
    for (int c = threadIdx.x; c < C; c += blockDim.x) rows[(size_t)v * C + c] = 0.f;
  }
}

// p and b of one token; s = 1 - a
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

DEVI float load_f(const float* p) { return *p; }
DEVI float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
DEVI void store_f(float* p, float v) { *p = v; }
DEVI void store_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16(v); }

template <int KIND>
DEVI void gate_grad(float g, float x, float p, float before, float lam, float& dg, float& dx) {
  if (KIND == TREE_GATE_SIGMOID) {
    const float s = lack(p);
    dx = lam * s;
    dg = dx * decay(p) * (before - x);
  } else {
    dx = lam;
    dg = g > 0.f ? 0.f : lam * decay(p) * before;
  }
}

template <typename T>
struct ScanFwd {
  const T *gate, *x;
  const float* init;
  T* y;
  float* states;
  const int32_t* tok_node;
  ScanLinks l;
  int N, n_nodes, C;
};

template <typename T>
struct ScanBwd {
  const T *gate, *x, *dy;
  const float *init, *states, *d_final;
  T *dgate, *dx;
  float* d_init;
  float *dnode, *before;
  const int32_t* tok_node;
  ScanLinks l;
  int N, n_nodes, C;
};

// One thread a channel, token by token.
template <typename T, int KIND>
__global__ void __launch_bounds__(64) k_scan_fwd(ScanFwd<T> a) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= a.C) return;
  float h = 0.f;
  for (int t = 0; t < a.N; ++t) {
    const int li = a.l.link[t];
    if (li == kLinkRoot) h = a.init ? a.init[(size_t)a.tok_node[t] * a.C + c] : 0.f;
    else if (li >= 0) h = a.states[(size_t)li * a.C + c];
    const size_t at = (size_t)t * a.C + c;
    float p, b;
    gate_of<KIND>(load_f(a.gate + at), load_f(a.x + at), p, b);
    h = scan_step(p, b, h);
    store_f(a.y + at, h);
    const int e = a.l.end[t];
    if (e >= 0) a.states[(size_t)e * a.C + c] = h;
    if (t % TILE == TILE - 1 || t == a.N - 1) a.states[(size_t)(a.n_nodes + t / TILE) * a.C + c] = h;
  }
}

template <typename T, int KIND>
__global__ void __launch_bounds__(64) k_scan_bwd(ScanBwd<T> a) {
  const int c = blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= a.C) return;
  float carry = 0.f;                                 // a lam of the token behind, if it follows on this path
  for (int k = (a.N - 1) / TILE; k >= 0; --k) {
    const int t0 = k * TILE, t1 = min(a.N, t0 + TILE);
    float h = k > 0 ? a.states[(size_t)(a.n_nodes + k - 1) * a.C + c] : 0.f;
    for (int t = t0; t < t1; ++t) {
      const int li = a.l.link[t];
      if (li == kLinkRoot) h = a.init ? a.init[(size_t)a.tok_node[t] * a.C + c] : 0.f;
      else if (li >= 0) h = a.states[(size_t)li * a.C + c];
      a.before[(size_t)(t - t0) * a.C + c] = h;
      const size_t at = (size_t)t * a.C + c;
      float p, b;
      gate_of<KIND>(load_f(a.gate + at), load_f(a.x + at), p, b);
      h = scan_step(p, b, h);
    }
    for (int t = t1 - 1; t >= t0; --t) {
      const size_t at = (size_t)t * a.C + c;
      float lam = load_f(a.dy + at) + carry;
      const int e = a.l.end[t];
      if (e >= 0 && a.d_final) lam += a.d_final[(size_t)e * a.C + c];
      if (a.l.kid[t] >= 0) lam += a.dnode[(size_t)a.l.kid[t] * a.C + c];
      const float g = load_f(a.gate + at), x = load_f(a.x + at);
      float p, b, dg, dx;
      gate_of<KIND>(g, x, p, b);
      gate_grad<KIND>(g, x, p, a.before[(size_t)(t - t0) * a.C + c], lam, dg, dx);
      store_f(a.dgate + at, dg);
      store_f(a.dx + at, dx);
      carry = scan_mul(p, lam);
      const int li = a.l.link[t];
      if (li != kLinkChain) {
        const int v = a.tok_node[t];
        if (li == kLinkRoot) {
          if (a.d_init) a.d_init[(size_t)v * a.C + c] = carry;
        } else {
          const float later = a.l.sib[t] >= 0 ? a.dnode[(size_t)a.l.sib[t] * a.C + c] : 0.f;
          a.dnode[(size_t)v * a.C + c] = carry + later;
        }
        carry = 0.f;
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// host side

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

struct ScanLayout {
  size_t link, end, kid, sib, dnode, before, total;
};

ScanLayout scan_layout(const tree_plan_t* p, int C) {
  ScanLayout L{};
  const size_t tok = align256((size_t)p->n_tokens * 4);
  size_t o = 0;
  L.link = o; o += tok;
  L.end = o;  o += tok;
  L.kid = o;  o += tok;
  L.sib = o;  o += tok;
  L.dnode = o;  o = align256(o + (size_t)p->n_nodes * C * 4);
  L.before = o; o = align256(o + (size_t)TILE * C * 4);
  L.total = o;
  return L;
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

ScanLinks links_at(void* workspace, const ScanLayout& L) {
  uint8_t* w = static_cast<uint8_t*>(workspace);
  return ScanLinks{reinterpret_cast<int32_t*>(w + L.link), reinterpret_cast<int32_t*>(w + L.end),
                   reinterpret_cast<int32_t*>(w + L.kid), reinterpret_cast<int32_t*>(w + L.sib)};
}

template <typename T, int KIND>
int run_fwd(const ScanFwd<T>& a, cudaStream_t s) {
  k_scan_fwd<T, KIND><<<(a.C + 63) / 64, 64, 0, s>>>(a);
  return record_cuda(cudaGetLastError());
}
template <typename T, int KIND>
int run_bwd(const ScanBwd<T>& a, cudaStream_t s) {
  k_scan_bwd<T, KIND><<<(a.C + 63) / 64, 64, 0, s>>>(a);
  return record_cuda(cudaGetLastError());
}

template <typename T>
int scan_fwd(const tree_plan_t* plan, const ScanLinks& l, const void* gate, const void* x, const float* init, int C,
             int kind, void* y, float* states, cudaStream_t s) {
  const ScanFwd<T> a{static_cast<const T*>(gate), static_cast<const T*>(x), init, static_cast<T*>(y), states,
                     plan->tok_node, l, plan->n_tokens, plan->n_nodes, C};
  return kind == TREE_GATE_SIGMOID ? run_fwd<T, TREE_GATE_SIGMOID>(a, s) : run_fwd<T, TREE_GATE_LOG>(a, s);
}

template <typename T>
int scan_bwd(const tree_plan_t* plan, const ScanLinks& l, const void* gate, const void* x, const float* init,
             const float* states, const void* dy, const float* d_final, int C, int kind, void* dgate, void* dx,
             float* d_init, float* dnode, float* before, cudaStream_t s) {
  const ScanBwd<T> a{static_cast<const T*>(gate), static_cast<const T*>(x), static_cast<const T*>(dy), init, states,
                     d_final, static_cast<T*>(dgate), static_cast<T*>(dx), d_init, dnode, before, plan->tok_node, l,
                     plan->n_tokens, plan->n_nodes, C};
  return kind == TREE_GATE_SIGMOID ? run_bwd<T, TREE_GATE_SIGMOID>(a, s) : run_bwd<T, TREE_GATE_LOG>(a, s);
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
  const ScanTree t{plan->tok_node, plan->tok_start, plan->sub_end, parent, node_len, plan->n_tokens, plan->n_nodes};
  const ScanLinks l = links_at(workspace, scan_layout(plan, C));
  k_scan_links<<<(unsigned)(((int64_t)t.N + 255) / 256), 256, 0, s>>>(t, l);
  k_scan_zero_rows<<<std::min(t.n_nodes, 152 * 8), 256, 0, s>>>(t, C, 0, states);
  rc = record_cuda(cudaGetLastError());
  if (rc) return rc;
  return dtype == TREE_BF16 ? scan_fwd<__nv_bfloat16>(plan, l, gate, x, init, C, gate_kind, y, states, s)
                            : scan_fwd<float>(plan, l, gate, x, init, C, gate_kind, y, states, s);
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
  const ScanTree t{plan->tok_node, plan->tok_start, plan->sub_end, parent, node_len, plan->n_tokens, plan->n_nodes};
  const ScanLayout L = scan_layout(plan, C);
  const ScanLinks l = links_at(workspace, L);
  uint8_t* w = static_cast<uint8_t*>(workspace);
  float* dnode = reinterpret_cast<float*>(w + L.dnode);
  float* before = reinterpret_cast<float*>(w + L.before);
  k_scan_links<<<(unsigned)(((int64_t)t.N + 255) / 256), 256, 0, s>>>(t, l);
  if (d_init) k_scan_zero_rows<<<std::min(t.n_nodes, 152 * 8), 256, 0, s>>>(t, C, 1, d_init);
  rc = record_cuda(cudaGetLastError());
  if (rc) return rc;
  return dtype == TREE_BF16
             ? scan_bwd<__nv_bfloat16>(plan, l, gate, x, init, states, dy, d_final, C, gate_kind, dgate, dx, d_init,
                                       dnode, before, s)
             : scan_bwd<float>(plan, l, gate, x, init, states, dy, d_final, C, gate_kind, dgate, dx, d_init, dnode,
                               before, s);
}

}  // extern "C"
