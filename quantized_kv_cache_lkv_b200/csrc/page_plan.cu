// page_plan.cu -- block tables, lengths and slot maps from request lengths
// (lkv_page_plan).
//
// need_b = ceil((len_b + new_b) / 256) - ceil(len_b / 256) pages; prefix sums
// of new_b and need_b over the sequences give every token its row and every
// new page its entry of the free stack, and cut the batch where the first
// sequence does not fit (both sums rise, so those that fit come first).
//
// Latency bound: a decode step moves a few hundred bytes.  So one launch, and
// no step that waits for another block: every block builds both prefix sums
// itself in shared memory (the lengths come out of L2), and a token on a new
// page takes the page from the free stack rather than from the table entry
// that some other block is writing.
#include <algorithm>

#include "serving.cuh"

namespace lkv {

namespace {

constexpr int kThreads = 512;

// Saturating sum of non-negative ints: past any capacity, but never wrapped.
__device__ __forceinline__ int add_sat(int a, int b) {
  const unsigned s = (unsigned)a + (unsigned)b;
  return s > 0x7FFFFFFFu ? 0x7FFFFFFF : (int)s;
}

__device__ __forceinline__ int pages_of(int tokens) { return (tokens + kPageTokens - 1) / kPageTokens; }

__device__ __forceinline__ bool sane(const PlanArgs& a, int len, int add) {
  return len >= 0 && add >= 0 && (long long)len + add <= (long long)a.pps * kPageTokens;
}

// Last b of [0, n) with first[b] <= x (first[0] = 0 <= x < first[n]).
__device__ __forceinline__ int owner(const int* first, int n, int x, int most) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (min(first[mid], most) <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// kRun: tokens of a thread and step.  Runs of four share a search and a page
// and store 16 bytes at a time (777 ragged requests, 583 thousand tokens: 9.7 us
// with runs of one, 6.6 with four); in a small call they only come one after the
// other (16 requests: 2.9 us with runs of one, 4.2 with four).
template <int kRun>
__global__ void __launch_bounds__(kThreads) page_plan_kernel(PlanArgs a) {
  extern __shared__ int s_tok[];       // [B + 1] tokens before each sequence
  int* s_pg = s_tok + a.B + 1;         // [B + 1] new pages before each sequence
  __shared__ int s_wt[32], s_wp[32], s_cut[2], s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int count = clamp_len(__ldg(a.free_count), a.free_cap);
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
  if (tid < 2) s_cut[tid] = 0;
  if (tid == 2) s_bad = 0;
  int nt = 0, np = 0;
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const int len = __ldg(a.lens + b), add = __ldg(a.n_new + b);
    const bool ok = sane(a, len, add);
    const int t = ok ? add : 0, p = ok ? pages_of(len + add) - pages_of(len) : 0;
    bad |= !ok;
    nt = add_sat(nt, t);
    np = add_sat(np, p);
    s_tok[b + 1] = nt;  // within the thread's run for now
    s_pg[b + 1] = np;
  }
  int it = nt, ip = np;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int x = __shfl_up_sync(0xFFFFFFFFu, it, off), y = __shfl_up_sync(0xFFFFFFFFu, ip, off);
    if (lane >= off) { it = add_sat(it, x); ip = add_sat(ip, y); }
  }
  if (lane == 31) { s_wt[warp] = it; s_wp[warp] = ip; }
  __syncthreads();
  // exclusive sums before this thread's run
  int et = __shfl_up_sync(0xFFFFFFFFu, it, 1), ep = __shfl_up_sync(0xFFFFFFFFu, ip, 1);
  if (lane == 0) et = ep = 0;
  for (int w = 0; w < warp; ++w) { et = add_sat(et, s_wt[w]); ep = add_sat(ep, s_wp[w]); }
  int ct = 0, cp = 0;
  for (int b = b0; b < b1; ++b) {
    const int t = add_sat(s_tok[b + 1], et), p = add_sat(s_pg[b + 1], ep);
    s_tok[b + 1] = t;
    s_pg[b + 1] = p;
    if (t <= a.n_cap && p <= count) { ct = t; cp = p; } else { bad = true; }
  }
  if (tid == 0) s_tok[0] = s_pg[0] = 0;
  if (ct) atomicMax(&s_cut[0], ct);
  if (cp) atomicMax(&s_cut[1], cp);
  if (bad) s_bad = 1;
  __syncthreads();
  // everything behind the cut counts as nothing: min() with these two
  const int tokens = s_cut[0], pages = s_cut[1];
  const int gt = blockIdx.x * kThreads + tid, gn = gridDim.x * kThreads;
  for (int b = gt; b < a.B; b += gn) {
    const int t0 = min(s_tok[b], tokens), t1 = min(s_tok[b + 1], tokens);
    a.new_lens[b] = __ldg(a.lens + b) + (t1 - t0);
    a.cu[b + 1] = t1;
  }
  for (int k = gt; k < pages; k += gn) {
    const int b = owner(s_pg, a.B, k, pages);
    const int j = pages_of(__ldg(a.lens + b)) + k - s_pg[b];
    a.table[(long long)b * a.pps + j] = __ldg(a.free_pages + count - 1 - k);
  }
  // runs of kRun tokens: one search each, and one page for as long as it lasts
  for (int r = gt; r < (tokens + kRun - 1) / kRun; r += gn) {
    const int t0 = r * kRun, t1 = min(tokens, t0 + kRun);
    int b = owner(s_tok, a.B, t0, tokens), next = t0, len = 0, old = 0, first = 0, base = 0, page = -1;
    int pos[kRun], seq[kRun];
    long long slot[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const int t = t0 + i;
      if (t < t1) {
        bool fresh = i == 0;
        if (i > 0 && t == next) {
          do ++b; while (min(s_tok[b + 1], tokens) <= t);  // past sequences without new tokens
          fresh = true;
        }
        if (fresh) {
          len = __ldg(a.lens + b);
          old = pages_of(len);
          first = s_tok[b];
          next = min(s_tok[b + 1], tokens);
          base = s_pg[b];
        }
        const int p = len + t - first, j = p / kPageTokens;
        if (fresh || p % kPageTokens == 0)
          page = j < old ? a.table[(long long)b * a.pps + j] : __ldg(a.free_pages + count - 1 - (base + j - old));
        pos[i] = p;
        seq[i] = b;
        slot[i] = page >= 0 && page < a.num_pages ? (long long)page * kPageTokens + p % kPageTokens : -1;
      }
    }
    if (kRun == 4 && t1 - t0 == kRun && a.wide) {
      *reinterpret_cast<int4*>(a.positions + t0) = make_int4(pos[0], pos[1 % kRun], pos[2 % kRun], pos[3 % kRun]);
      *reinterpret_cast<int4*>(a.token_seq + t0) = make_int4(seq[0], seq[1 % kRun], seq[2 % kRun], seq[3 % kRun]);
      *reinterpret_cast<longlong2*>(a.slots + t0) = make_longlong2(slot[0], slot[1 % kRun]);
      *reinterpret_cast<longlong2*>(a.slots + t0 + 2) = make_longlong2(slot[2 % kRun], slot[3 % kRun]);
    } else {
#pragma unroll
      for (int i = 0; i < kRun; ++i)
        if (t0 + i < t1) {
          a.positions[t0 + i] = pos[i];
          a.token_seq[t0 + i] = seq[i];
          a.slots[t0 + i] = slot[i];
        }
    }
  }
  if (blockIdx.x != gridDim.x - 1) return;
  // the last block also answers for the call: every page a new token can lie
  // on is a taken one or the last old page of a served sequence
  if (tid == 0) { a.cu[0] = 0; a.free_left[0] = count - pages; }
  if (a.status == nullptr) return;
  bad = false;
  for (int k = tid; k < pages; k += kThreads) {
    const int page = __ldg(a.free_pages + count - 1 - k);
    bad |= page < 0 || page >= a.num_pages;
  }
  for (int b = tid; b < a.B; b += kThreads) {
    const int len = __ldg(a.lens + b);
    if (min(s_tok[b + 1], tokens) > min(s_tok[b], tokens) && len % kPageTokens != 0) {
      const int page = a.table[(long long)b * a.pps + len / kPageTokens];
      bad |= page < 0 || page >= a.num_pages;
    }
  }
  if (bad) s_bad = 1;
  __syncthreads();
  if (tid == 0) a.status[0] = s_bad ? kStatusInvalidArg : 0;
}

}  // namespace

template <int kRun>
static cudaError_t launch_run(const PlanArgs& a, cudaStream_t s) {
  const size_t smem = (size_t)2 * (a.B + 1) * sizeof(int);
  if (smem > 48 * 1024) {
    // the kernel's limit, not this call's: calls of other batches from other threads set the same
    const cudaError_t e = cudaFuncSetAttribute(page_plan_kernel<kRun>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               2 * (kPlanMaxBatch + 1) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
  }
  const long long want = (std::max((long long)a.n_cap / kRun + 1, (long long)a.B) + kThreads - 1) / kThreads;
  const int grid = (int)std::max<long long>(1, std::min<long long>(num_sms(), want));
  page_plan_kernel<kRun><<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_page_plan(const PlanArgs& a, cudaStream_t s) {
  // a token per thread while one wave of blocks covers the capacity (how many there are, the host does not know)
  return a.n_cap <= num_sms() * kThreads ? launch_run<1>(a, s) : launch_run<4>(a, s);
}

}  // namespace lkv
