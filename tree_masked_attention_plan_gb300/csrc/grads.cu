// Global gradient norm over a list of tensors, and clipping by it.
//   norm = sqrt(sum over all tensors and elements of g^2),
//   out  = g * (max_norm / norm) where max_norm < norm < inf, else g.
// HBM-bound: the norm reads every gradient once; clipping reads it again and writes it.  218M bf16 elements are
// clipped in 0.216 ms, 528M fp32 in 0.95 ms (6.1 and 6.7 TB/s of three times their bytes); the norm of 291 small
// tensors, 6 MB, takes 7.3 us, of which two launches are most.
// The list travels in the kernel's parameters, so a call copies nothing to the device and can be
// captured.  Work is dealt out in chunks of kChunk elements, each inside one tensor.
// Determinism: a block's chunks, a thread's elements and the order of every sum depend on the list
// alone, and no atomics are used: the same gradients give the same norm, bit for bit.
#include <algorithm>
#include <cmath>
#include <vector>

#include "common.cuh"

namespace ta {
namespace {

constexpr int kChunk = 16384;                 // elements of a unit of work: 32 or 64 KB read
constexpr int kGradThreads = 256;
constexpr int kGradBlocks = 152 * 8;          // most blocks of a launch, and partial sums of one

struct GradEntry {
  const uint8_t* src;
  uint8_t* dst;
  int64_t numel;
  int32_t first;                              // first chunk of the tensor
  int32_t f32;
};

// Lists longer than kLongList take several launches of each kind.  Short ones travel in a kernel of fewer parameters:
// the GPU takes 24 KB of them at a time only as kernels end, so that calls of 12 tensors each, 218M elements, would
// come back after 137 us instead of 13.
constexpr int kSmallList = 64, kLongList = 768;

template <int MAX>
struct GradList {
  GradEntry e[MAX];
  int n, chunks;
};

// A thread's sum of squares.  fp64 additions are rare on this GPU (two a clock and SM: one for every 16-byte
// vector made the norm of 528M fp32 elements take 2.4 ms instead of 0.3), so a vector's squares are summed in
// fp32 and the vectors' sums in a pair of fp32 that holds what each addition rounds away.  A vector with a value
// above 2^40 or with none above 2^-50, whose squares fp32 may not hold, is squared and summed in fp64.
// A vector's sum takes 4 roundings (fp32) or 7 (bf16, whose squares are exact), the pair by the time that it holds as many
// equal values as fit the memory 7 more: 7 units of 2^-24 in the norm, and its own rounding.
struct Squares {
  float s = 0.f, c = 0.f;
  double rest = 0.0;
  DEVI void add(float v) {                    // s + c += v: s takes the rounded sum, c the rounding
    const float t = s + v, z = t - s;
    c += (s - (t - z)) + (v - z);
    s = t;
  }
  template <int CNT>
  DEVI void vec(const float (&v)[CNT]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < CNT; ++i) m = fmaxf(m, fabsf(v[i]));
    if (m > 0x1p40f || (m < 0x1p-50f && m > 0.f)) {
#pragma unroll
      for (int i = 0; i < CNT; ++i) rest += (double)v[i] * (double)v[i];
    } else {
      float q = 0.f;
#pragma unroll
      for (int i = 0; i < CNT; ++i) q = fmaf(v[i], v[i], q);
      add(q);
    }
  }
};

DEVI void load_vec(const uint8_t* p, float (&v)[4]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
DEVI void load_vec(const uint8_t* p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16lo(w[i]);
    v[2 * i + 1] = bf16hi(w[i]);
  }
}
DEVI void store_vec(uint8_t* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
DEVI void store_vec(uint8_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                            pack_bf16(v[6], v[7]));
}
template <int CNT>
DEVI float load_one(const uint8_t* p) {
  if (CNT == 4) return *reinterpret_cast<const float*>(p);
  return __uint_as_float(static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << 16);
}
template <int CNT>
DEVI void store_one(uint8_t* p, float v) {
  if (CNT == 4) *reinterpret_cast<float*>(p) = v;
  else *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16(v);
}

// elements before p's next 16-byte boundary
template <int CNT>
DEVI int64_t head_elems(const uint8_t* p, int64_t n) {
  const int64_t h = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / (16 / CNT);
  return h < n ? h : n;
}

// one chunk's n elements at p, this thread's share
template <int CNT>
DEVI void chunk_squares(const uint8_t* p, int64_t n, Squares& sq) {
  constexpr int ES = 16 / CNT;
  const int64_t head = head_elems<CNT>(p, n);
  const int nvec = static_cast<int>((n - head) / CNT);
  const uint8_t* pv = p + head * ES;
  int i = threadIdx.x;
  for (; i + 3 * kGradThreads < nvec; i += 4 * kGradThreads) {       // four loads in flight
    float v[4][CNT];
#pragma unroll
    for (int q = 0; q < 4; ++q) load_vec(pv + (size_t)(i + q * kGradThreads) * 16, v[q]);
#pragma unroll
    for (int q = 0; q < 4; ++q) sq.vec(v[q]);
  }
  for (; i < nvec; i += kGradThreads) {
    float v[CNT];
    load_vec(pv + (size_t)i * 16, v);
    sq.vec(v);
  }
  const int64_t tail = head + (int64_t)nvec * CNT;
  const int64_t rest = head + (n - tail);          // single elements: before and behind the vectors
  if (threadIdx.x < rest) {
    const int64_t j = threadIdx.x < head ? threadIdx.x : tail + (threadIdx.x - head);
    const float one[1] = {load_one<CNT>(p + j * ES)};
    sq.vec(one);
  }
}

// the block's sum, in thread 0
DEVI double block_squares(Squares& q, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float s = __shfl_xor_sync(0xffffffffu, q.s, o), c = __shfl_xor_sync(0xffffffffu, q.c, o);
    q.add(s);
    q.c += c;
  }
  double v = (double)q.s + (double)q.c;
  if (__any_sync(0xffffffffu, q.rest != 0.0)) {    // (NaN: the sum is NaN)
    double r = q.rest;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    v += r;
  }
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < kGradThreads / 32; ++i) s += red[i];
  return s;
}

DEVI double block_sum(double v, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kGradThreads / 32; ++i) s += red[i];
  return s;
}

// the entry that holds chunk c: the last one whose first chunk is not behind it and that has any
template <int MAX>
DEVI int entry_of(const GradList<MAX>& L, int c) {
  int lo = 0, hi = L.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (L.e[mid].first <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int MAX>
__global__ void __launch_bounds__(kGradThreads) k_grad_squares(const __grid_constant__ GradList<MAX> L, double* part) {
  __shared__ double red[kGradThreads / 32];
  Squares sq;
  for (int c = blockIdx.x; c < L.chunks; c += gridDim.x) {
    const GradEntry& e = L.e[entry_of(L, c)];
    const int64_t at = (int64_t)(c - e.first) * kChunk;
    const int64_t n = min((int64_t)kChunk, e.numel - at);
    if (e.f32) chunk_squares<4>(e.src + at * 4, n, sq);
    else chunk_squares<8>(e.src + at * 2, n, sq);
  }
  const double s = block_squares(sq, red);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// the sum of the n partial sums, in an order that depends on n alone; every thread gets it
DEVI double total_squares(const double* part, int n, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kGradThreads) s += part[i];
  return block_sum(s, red);
}

__global__ void __launch_bounds__(kGradThreads) k_grad_norm(const double* part, int n, float* norm) {
  __shared__ double red[kGradThreads / 32];
  const double s = total_squares(part, n, red);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(s));
}

// one chunk from p to o: scaled, or where CLIP is false copied bit by bit (a NaN keeps its payload)
template <int CNT, bool CLIP>
DEVI void chunk_scale(const uint8_t* p, uint8_t* o, int64_t n, float c) {
  constexpr int ES = 16 / CNT;
  auto one = [&](int64_t i) {
    if (CLIP) store_one<CNT>(o + i * ES, c * load_one<CNT>(p + i * ES));
    else if (CNT == 4) *reinterpret_cast<uint32_t*>(o + i * ES) = *reinterpret_cast<const uint32_t*>(p + i * ES);
    else *reinterpret_cast<uint16_t*>(o + i * ES) = *reinterpret_cast<const uint16_t*>(p + i * ES);
  };
  if ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) {
    // source and target differ in their place within 16 bytes: element by element
    for (int64_t i = threadIdx.x; i < n; i += kGradThreads) one(i);
    return;
  }
  const int64_t head = head_elems<CNT>(p, n);
  const int nvec = static_cast<int>((n - head) / CNT);
  auto out = [&](uint8_t* to, uint4 w) {
    if (CLIP) {
      float v[CNT];
      load_vec(reinterpret_cast<const uint8_t*>(&w), v);
#pragma unroll
      for (int e = 0; e < CNT; ++e) v[e] *= c;
      store_vec(to, v);
    } else {
      *reinterpret_cast<uint4*>(to) = w;
    }
  };
  const uint8_t* pv = p + head * ES;
  uint8_t* ov = o + head * ES;
  int i = threadIdx.x;
  for (; i + 3 * kGradThreads < nvec; i += 4 * kGradThreads) {
    uint4 w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = *reinterpret_cast<const uint4*>(pv + (size_t)(i + q * kGradThreads) * 16);
#pragma unroll
    for (int q = 0; q < 4; ++q) out(ov + (size_t)(i + q * kGradThreads) * 16, w[q]);
  }
  for (; i < nvec; i += kGradThreads) out(ov + (size_t)i * 16, *reinterpret_cast<const uint4*>(pv + (size_t)i * 16));
  const int64_t tail = head + (int64_t)nvec * CNT;
  const int64_t rest = head + (n - tail);
  if (threadIdx.x < rest) one(threadIdx.x < head ? threadIdx.x : tail + (threadIdx.x - head));
}

template <int CNT>
DEVI void chunk_out(const uint8_t* p, uint8_t* o, int64_t n, bool clip, float c) {
  if (clip) chunk_scale<CNT, true>(p, o, n, c);
  else if (p != o) chunk_scale<CNT, false>(p, o, n, c);
}

// Every block adds the partial sums up for itself (a few KB from L2) and scales its chunks, the
// last ones first: they are the ones that the norm's pass left in L2.
template <int MAX>
__global__ void __launch_bounds__(kGradThreads) k_grad_scale(const __grid_constant__ GradList<MAX> L,
                                                             const double* part, int n_part, double max_norm,
                                                             float* norm) {
  __shared__ double red[kGradThreads / 32];
  const double total = sqrt(total_squares(part, n_part, red));
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  const bool clip = total > max_norm && (float)total < INFINITY;      // false for NaN
  const float coef = clip ? static_cast<float>(max_norm / total) : 1.f;
  for (int c = L.chunks - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
    const GradEntry& e = L.e[entry_of(L, c)];
    const int64_t at = (int64_t)(c - e.first) * kChunk;
    const int64_t n = min((int64_t)kChunk, e.numel - at);
    if (e.f32) chunk_out<4>(e.src + at * 4, e.dst + at * 4, n, clip, coef);
    else chunk_out<8>(e.src + at * 2, e.dst + at * 2, n, clip, coef);
  }
}

int64_t grad_bytes(const tree_grad_t& g) { return g.numel * (g.dtype == TREE_F32 ? 4 : 2); }

int check_list(const tree_grad_t* list, int n, bool clip) {
  if (!list) return TREE_ERR_ARG;
  if (n <= 0) return TREE_ERR_SHAPE;
  int64_t chunks = 0;
  for (int i = 0; i < n; ++i) {
    const tree_grad_t& g = list[i];
    if (g.numel < 0 || (g.dtype != TREE_BF16 && g.dtype != TREE_F32)) return TREE_ERR_SHAPE;
    if (g.numel > 0 && (!g.grad || (clip && !g.out))) return TREE_ERR_ARG;
    const uintptr_t mask = g.dtype == TREE_F32 ? 3 : 1;
    if ((reinterpret_cast<uintptr_t>(g.grad) | (clip ? reinterpret_cast<uintptr_t>(g.out) : 0)) & mask)
      return TREE_ERR_ARG;
    if (g.numel > ((int64_t)1 << 44)) return TREE_ERR_SHAPE;
    chunks += (g.numel + kChunk - 1) / kChunk;
  }
  if (chunks > 0x7fffffff) return TREE_ERR_SHAPE;
  if (!clip) return TREE_OK;
  // No target may touch another one, nor a gradient other than its own, which it may only equal.
  struct Span {
    uintptr_t lo, hi;
    bool out;
  };
  std::vector<Span> v;
  try {
    v.reserve(2 * (size_t)n);
  } catch (...) {                            // no exception crosses the C boundary
    return TREE_ERR_ARG;
  }
  for (int i = 0; i < n; ++i) {
    const int64_t b = grad_bytes(list[i]);
    if (!b) continue;
    const uintptr_t s = reinterpret_cast<uintptr_t>(list[i].grad), o = reinterpret_cast<uintptr_t>(list[i].out);
    v.push_back({o, o + (uintptr_t)b, true});
    if (s != o) v.push_back({s, s + (uintptr_t)b, false});
  }
  std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uintptr_t end_any = 0, end_out = 0;        // the furthest end so far, and that of a target
  for (const Span& a : v) {
    if (a.lo < (a.out ? end_any : end_out)) return TREE_ERR_ARG;
    end_any = std::max(end_any, a.hi);
    if (a.out) end_out = std::max(end_out, a.hi);
  }
  return TREE_OK;
}

template <int MAX>
void fill(GradList<MAX>* L, const tree_grad_t* list, int n) {
  int m = 0, chunks = 0;
  for (int i = 0; i < n; ++i) {
    if (list[i].numel == 0) continue;
    L->e[m++] = GradEntry{static_cast<const uint8_t*>(list[i].grad), static_cast<uint8_t*>(list[i].out),
                          list[i].numel, chunks, list[i].dtype == TREE_F32};
    chunks += static_cast<int>((list[i].numel + kChunk - 1) / kChunk);
  }
  L->n = m;
  L->chunks = chunks;
}

template <int MAX>
int squares_of(const tree_grad_t* list, int n, double* part, int* blocks, cudaStream_t s) {
  GradList<MAX> L;
  fill(&L, list, n);
  *blocks = std::min(L.chunks, kGradBlocks);
  if (*blocks == 0) return TREE_OK;
  k_grad_squares<MAX><<<*blocks, kGradThreads, 0, s>>>(L, part);
  return record_cuda(cudaGetLastError());
}

template <int MAX>
int scale_by(const tree_grad_t* list, int n, const double* part, int n_part, double max_norm, float* norm,
             cudaStream_t s) {
  GradList<MAX> L;
  fill(&L, list, n);
  k_grad_scale<MAX><<<std::max(1, std::min(L.chunks, kGradBlocks)), kGradThreads, 0, s>>>(L, part, n_part, max_norm,
                                                                                         norm);
  return record_cuda(cudaGetLastError());
}

// the partial sums of the whole list, kLongList tensors a launch
int all_squares(const tree_grad_t* list, int n, double* part, int* n_part, cudaStream_t s) {
  *n_part = 0;
  for (int i = 0; i < n; i += kLongList) {
    const int m = std::min(kLongList, n - i);
    int blocks = 0;
    const int rc = m <= kSmallList ? squares_of<kSmallList>(list + i, m, part + *n_part, &blocks, s)
                                   : squares_of<kLongList>(list + i, m, part + *n_part, &blocks, s);
    if (rc) return rc;
    *n_part += blocks;
  }
  return TREE_OK;
}

bool bad_ws(const void* p) { return !p || (reinterpret_cast<uintptr_t>(p) & 15); }

// Partial sums and the norm are written while other blocks read gradients and write targets: they touch none, nor each other.
bool results_apart(const tree_grad_t* list, int n, bool clip, const void* workspace, const float* norm) {
  const size_t ws = tree_grad_workspace(n);
  if (buffers_meet(workspace, ws, norm, 4)) return false;
  for (int i = 0; i < n; ++i) {
    const size_t b = (size_t)grad_bytes(list[i]);
    if (!b) continue;
    for (const void* p : {list[i].grad, clip ? static_cast<const void*>(list[i].out) : nullptr})
      if (buffers_meet(p, b, workspace, ws) || buffers_meet(p, b, norm, 4)) return false;
  }
  return true;
}

}  // namespace
}  // namespace ta

using namespace ta;

extern "C" {

size_t tree_grad_workspace(int n) {
  if (n <= 0) return 0;
  return (size_t)((n + kLongList - 1) / kLongList) * kGradBlocks * sizeof(double);
}

int tree_grad_norm(const tree_grad_t* list, int n, void* workspace, float* norm, tree_stream_t stream) {
  int rc = check_list(list, n, false);
  if (rc) return rc;
  if (bad_ws(workspace) || !norm || (reinterpret_cast<uintptr_t>(norm) & 3)) return TREE_ERR_ARG;
  if (!results_apart(list, n, false, workspace, norm)) return TREE_ERR_ARG;
  rc = check_device();
  if (rc) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  int n_part = 0;
  rc = all_squares(list, n, part, &n_part, s);
  if (rc) return rc;
  k_grad_norm<<<1, kGradThreads, 0, s>>>(part, n_part, norm);
  return record_cuda(cudaGetLastError());
}

int tree_grad_clip(const tree_grad_t* list, int n, double max_norm, void* workspace, float* norm,
                   tree_stream_t stream) {
  int rc = check_list(list, n, true);
  if (rc) return rc;
  if (!(max_norm >= 0.0)) return TREE_ERR_SHAPE;
  if (bad_ws(workspace) || !norm || (reinterpret_cast<uintptr_t>(norm) & 3)) return TREE_ERR_ARG;
  if (!results_apart(list, n, true, workspace, norm)) return TREE_ERR_ARG;
  rc = check_device();
  if (rc) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  int n_part = 0;
  rc = all_squares(list, n, part, &n_part, s);
  if (rc) return rc;
  for (int i = 0; i < n; i += kLongList) {
    const int m = std::min(kLongList, n - i);
    rc = m <= kSmallList ? scale_by<kSmallList>(list + i, m, part, n_part, max_norm, norm, s)
                         : scale_by<kLongList>(list + i, m, part, n_part, max_norm, norm, s);
    if (rc) return rc;
  }
  return TREE_OK;
}

}  // extern "C"
