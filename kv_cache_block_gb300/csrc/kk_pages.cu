// Pages with reference counts: taken, given back, forked and compacted
// (kk_pages_alloc, kk_pages_free, kk_pages_fork, kk_pages_compact).
//
// What is to be done is planned on the device, so that a beam search's step
// needs no word from the host: one cluster of up to eight CTAs goes through the
// tables and counts in phases that a cluster barrier separates (a few
// microseconds, where a launch a phase would cost each of them its latency), and
// leaves a list of (from, to) pages; small pools are planned by one CTA in its
// shared memory. The copies, the part that moves bytes, follow in a launch that
// fills the GPU: 231 pages of 7.3 MB (3.4 GB read and written) 538 us, 6.3 TB/s; with four blocks an SM
// (64 registers, spilled) 567, with loads of one slice at a time 545. Counts change by integer atomics and free pages
// are taken in ascending order: the result does not depend on timing.
#include "kk_pages.cuh"

#include <algorithm>
#include <climits>

#include "kk_attn.cuh"
#include "kk_pdl.cuh"

namespace kk {
namespace {

constexpr int kPlan = 1024;       // threads of a planning CTA
constexpr int kPlanCtas = 8;      // CTAs of the planning cluster, at most
constexpr int kStep = kPlan * 4;  // counts a CTA looks at in a turn

__device__ __forceinline__ void cluster_sync() {
  __threadfence();
  cluster_arrive_release();
  cluster_wait_acquire();
}
struct Place {  // of a thread in the planning cluster
  int cta, ctas, tid, all, n;  // its number among all n threads
};
__device__ __forceinline__ Place place() {
  pdl_wait();  // what ran before in the stream has finished; what comes next may be launched
  pdl_launch_dependents();
  Place p;
  p.cta = (int)cluster_rank();
  p.ctas = (int)cluster_size();
  p.tid = threadIdx.x;
  p.all = p.cta * kPlan + p.tid;
  p.n = p.ctas * kPlan;
  return p;
}

// Exclusive sum of x over the CTA's threads; *total gets the sum. `sh`: 33 ints.
__device__ __forceinline__ int block_scan(int x, int* sh, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();
  if (lane == 31) sh[w] = v;
  __syncthreads();
  if (w == 0) {
    int y = sh[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(kFull, y, o);
      if (lane >= o) y += z;
    }
    sh[lane] = y;
  }
  __syncthreads();
  *total = sh[31];
  return v - x + (w ? sh[w - 1] : 0);
}

// The same integer of every CTA of the cluster, summed over those before this one and over all.
// `box`: kPlanCtas ints of shared memory, not used again before the next cluster barrier but one.
__device__ __forceinline__ void cluster_sums(int mine, int* box, const Place& p, int* before, int* total) {
  if (p.tid < p.ctas) st_cluster_s32(map_to_rank(smem_u32(box + p.cta), (uint32_t)p.tid), mine);
  cluster_arrive_release();
  cluster_wait_acquire();
  int b = 0, t = 0;
  for (int c = 0; c < p.ctas; ++c) {
    if (c < p.cta) b += box[c];
    t += box[c];
  }
  *before = b;
  *total = t;
}

__device__ __forceinline__ void copy_refs(const int* in, int* out, int n, const Place& p) {
  if (in == out) return;
  for (int i = p.all; i < n; i += p.n) out[i] = in[i];
}

// Calls take(k, page) for the k-th free page in ascending order, k < need; returns how many there were, at most
// `need`. All threads of the cluster call it. Reads counts past L1: they change during the kernel.
template <typename F>
__device__ __forceinline__ int take_free(const int* refs, int pages, int need, const Place& p, int* sh, int* box,
                                         F take) {
  int found = 0;
  for (long long at = 0, turn = 0; at < pages && found < need; at += (long long)p.ctas * kStep, turn ^= 1) {
    const long long i0 = at + (long long)p.cta * kStep + p.tid * 4;
    int free4 = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i0 + e < pages && __ldcg(refs + i0 + e) == 0) free4 |= 1 << e;
    int mine, before, total;
    int k = block_scan(__popc(free4), sh, &mine);
    cluster_sums(mine, box + turn * kPlanCtas, p, &before, &total);
    k += found + before;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (free4 >> e & 1) {
        if (k < need) take(k, (int)(i0 + e));
        ++k;
      }
    found += total;
  }
  return min(found, need);
}

// Warps [first, n) of the cluster share out the items of x < count, each item's `parts` warps having a part of
// it: calls f(item, first element of the lane, step).
template <typename F>
__device__ __forceinline__ void share_warps(int wid, int n, int count, F f) {
  if (wid < 0 || count <= 0) return;
  const int parts = max(1, n / count), lane = threadIdx.x & 31;
  for (long long x = wid; x < (long long)count * parts; x += n)
    f((int)(x / parts), (int)(x % parts) * 32 + lane, parts * 32);
}

__global__ void __launch_bounds__(kPlan) pages_free_kernel(Table bt, const int* refs_in, int* refs_out, int pages,
                                                           int* err) {
  const Place p = place();
  copy_refs(refs_in, refs_out, pages, p);
  if (refs_in != refs_out) cluster_sync();
  share_warps(p.all >> 5, p.n >> 5, bt.R, [&](int r, int j0, int step) {
    const int off = bt.offsets[r], nb = bt.offsets[r + 1] - off;
    if (nb < 0 || nb > bt.max_blocks) {
      flag_error(err, kErrBadIndex);
      return;
    }
    for (int j = j0; j < nb; j += step) {
      const int page = bt.pages[off + j];
      if (page < 0 || page >= pages) {
        flag_error(err, kErrBadIndex);
      } else if (atomicSub(refs_out + page, 1) <= 0) {  // was free: as many succeed as there were counts
        atomicAdd(refs_out + page, 1);
        flag_error(err, kErrBadIndex);
      }
    }
  });
}

__global__ void __launch_bounds__(kPlan) pages_alloc_kernel(const int* refs_in, int* refs_out, int pages,
                                                            const int* want, int n, int* out, int* err) {
  __shared__ int sh[33], box[2 * kPlanCtas];
  const Place p = place();
  copy_refs(refs_in, refs_out, pages, p);
  int need = n;
  if (want) {  // every CTA counts for itself
    int mine = 0;
    for (int i = p.tid; i < n; i += kPlan) mine += want[i] != 0;
    int total;
    block_scan(mine, sh, &total);
    need = total;
  }
  cluster_sync();
  // pages in the order of the takers first: taker k's page at out[k]
  const int got = take_free(refs_out, pages, need, p, sh, box, [&](int k, int page) {
    refs_out[page] = 1;
    out[k] = page;
  });
  cluster_sync();
  if (p.cta) return;
  if (got < need && p.tid == 0) flag_error(err, kErrNoPages);
  // then to the takers' places, the last ones first: taker k's place is not before k, so what is still to be
  // read lies in front of everything written
  int left = need;
  for (int c = (n + kPlan - 1) / kPlan - 1; c >= 0; --c) {
    const int i = c * kPlan + p.tid;
    const bool takes = i < n && (!want || want[i] != 0);
    int total;
    const int k = left + block_scan(takes ? 1 : 0, sh, &total) - total;
    left -= total;
    const int page = takes && k < got ? __ldcg(out + k) : -1;
    __syncthreads();
    if (i < n) out[i] = page;
    __syncthreads();
  }
}

// A parent as its children take it; n < 0: its table disagrees with its length.
struct Parent {
  int off, n, T;
  bool part;  // its last block is not full
};
__device__ __forceinline__ Parent parent_of(const ForkArgs& a, int r) {
  Parent x;
  x.off = a.bt.offsets[r];
  x.n = a.bt.offsets[r + 1] - x.off;
  x.T = a.bt.seq_lens[r];
  if (x.T < 0 || x.T > kMaxTokens || x.n < 0 || x.n > a.bt.max_blocks ||
      x.n != (int)(((unsigned)x.T + (unsigned)a.bs - 1u) / (unsigned)a.bs))
    x.n = -1;
  x.part = x.n > 0 && x.T % a.bs != 0;
  return x;
}

// How a fork changes the count of a page for a place it has in a parent's table: the open block's (`open`), or another.
__device__ __forceinline__ int change_of(const ForkArgs& a, int kids, bool open) {
  return open ? (a.keep ? 0 : (kids ? 0 : -1)) : (a.keep ? kids : kids - 1);
}

// Counts that were missing. A table's own count is there until its change, whatever the others do, so a change finds
// 0 only where tables have more places than the page has counts. The changes are then taken back and made
// again by make_count, in three passes over the tables: a count of 0 becomes kMissing plus the places that hold the page
// afterwards, in whatever order the tables come, and real_count says what that is.
constexpr int kMissing = -(1 << 30);
__device__ __forceinline__ void make_count(int* at, int more) {
  int c = 0;
  for (;;) {
    const int seen = atomicCAS(at, c, c > 0 ? c + more : (c < kMissing / 2 ? c : kMissing) + more + 1);
    if (seen == c) return;
    c = seen;
  }
}
__device__ __forceinline__ int real_count(int c) { return c >= 0 ? c : max(0, c < kMissing / 2 ? c - kMissing : 0); }

__global__ void __launch_bounds__(kPlan) pages_fork_kernel(const ForkArgs a) {
  __shared__ int sh[33], box[2 * kPlanCtas];
  const Place p = place();
  copy_refs(a.refs_in, a.refs_out, a.num_pages, p);
  for (int r = p.all; r < a.bt.R; r += p.n) {
    a.kids[r] = 0;
    a.first[r] = INT_MAX;
  }
  int* missing = a.n_pairs + 1;  // whether a place in a table had no count
  if (p.all == 0) *missing = 0;
  cluster_sync();
  for (int i = p.all; i < a.F; i += p.n) {
    const int r = a.parent[i];
    const bool ok = r >= 0 && r < a.bt.R && parent_of(a, r).n >= 0;
    if (!ok) {
      flag_error(a.err, kErrBadIndex);
      continue;
    }
    atomicAdd(a.kids + r, 1);
    atomicMin(a.first + r, i);
  }
  cluster_sync();
  // CTA 0 lays the children out, the others (or it, alone) move the counts
  if (p.cta == 0) {
    int off = 0, copies = 0;
    for (int i0 = 0; i0 < a.F; i0 += kPlan) {
      const int i = i0 + p.tid;
      int r = -1, n = 0, T = 0, last = 0;
      bool copy = false;
      if (i < a.F) {
        r = a.parent[i];
        if (r >= 0 && r < a.bt.R) {
          const Parent x = parent_of(a, r);
          if (x.n >= 0) {
            n = x.n;
            T = x.T;
            copy = x.part && (a.keep || __ldcg(a.first + r) != i);
            if (copy) last = a.bt.pages[x.off + n - 1];
          }
        }
      }
      int total;
      const int to = off + block_scan(n, sh, &total);
      off += total;
      const int k = copies + block_scan(copy ? 1 : 0, sh, &total);
      copies += total;
      if (i < a.F) {
        a.child_offsets[i] = to;
        a.child_lens[i] = T;
        if (copy) {
          a.pairs[k] = make_int2(last, -1);
          a.at[k] = to + n - 1;
        }
      }
    }
    if (p.tid == 0) {
      a.child_offsets[a.F] = off;
      a.at[a.F] = copies;
    }
  }
  const int lead = p.ctas > 1 ? kPlan / 32 : 0;  // CTA 0's warps stay out
  auto places = [&](auto f) {  // f(page, change) for every place of a page in the tables; a page out of range is reported
    share_warps((p.all >> 5) - lead, (p.n >> 5) - lead, a.bt.R, [&](int r, int j0, int step) {
      const Parent x = parent_of(a, r);
      const int kids = __ldcg(a.kids + r);
      if (x.n < 0 && !a.keep && j0 == 0) flag_error(a.err, kErrBadIndex);  // its counts cannot be given back
      for (int j = j0; j < x.n; j += step) {
        const int page = a.bt.pages[x.off + j];
        if (page < 0 || page >= a.num_pages) flag_error(a.err, kErrBadIndex);
        else f(page, change_of(a, kids, j == x.n - 1 && x.part));
      }
    });
  };
  places([&](int page, int more) {
    const int had = more ? atomicAdd(a.refs_out + page, more) : __ldcg(a.refs_out + page);
    if (had <= 0) {
      *missing = 1;
      flag_error(a.err, kErrBadIndex);
    }
  });
  cluster_sync();
  const bool mend = __ldcg(missing) != 0;  // the same for the cluster
  share_warps(p.all >> 5, p.n >> 5, a.F, [&](int i, int j0, int step) {
    const int to = __ldcg(a.child_offsets + i), n = __ldcg(a.child_offsets + i + 1) - to;
    if (n == 0) return;
    const int r = a.parent[i];
    const Parent x = parent_of(a, r);
    const bool copy = x.part && (a.keep || __ldcg(a.first + r) != i);
    for (int j = j0; j < n - (copy ? 1 : 0); j += step) a.child_pages[to + j] = a.bt.pages[x.off + j];
  });
  if (mend) {
    places([&](int page, int more) { atomicSub(a.refs_out + page, more); });
    cluster_sync();
    places([&](int page, int more) { make_count(a.refs_out + page, more); });
    cluster_sync();
    for (int i = p.all; i < a.num_pages; i += p.n) {
      const int c = __ldcg(a.refs_out + i);
      if (c < 0) a.refs_out[i] = real_count(c);
    }
    cluster_sync();
  }
  const int need = __ldcg(a.at + a.F);
  const int got = take_free(a.refs_out, a.num_pages, need, p, sh, box, [&](int k, int page) {
    a.refs_out[page] = 1;
    a.pairs[k].y = page;
    a.child_pages[__ldcg(a.at + k)] = page;
  });
  for (int k = got + p.all; k < need; k += p.n) a.child_pages[__ldcg(a.at + k)] = -1;
  if (p.all == 0) {
    *a.n_pairs = got;
    if (got < need) flag_error(a.err, kErrNoPages);
  }
}

__global__ void __launch_bounds__(kPlan) pages_compact_kernel(const CompactArgs a) {
  __shared__ int sh[33], box[2 * kPlanCtas];
  const Place p = place();
  cluster_sync();  // every CTA of the cluster runs before another writes to its shared memory
  // a CTA's share of the pages, in order
  const long long per = ((long long)a.num_pages + p.ctas - 1) / p.ctas;
  const int lo = (int)min((long long)a.num_pages, per * p.cta);
  const int hi = (int)min((long long)a.num_pages, per * (p.cta + 1));
  int mine = 0, total, before, used;
  for (int i = lo + p.tid; i < hi; i += kPlan) mine += a.refs_in[i] != 0;
  block_scan(mine, sh, &total);
  cluster_sums(total, box, p, &before, &used);
  // `before`: used pages in front of the share; those below `used` stay
  mine = 0;
  for (int i = lo + p.tid; i < min(hi, used); i += kPlan) mine += a.refs_in[i] != 0;
  block_scan(mine, sh, &total);
  int dummy, stay;
  cluster_sums(total, box + kPlanCtas, p, &dummy, &stay);
  const int moves = used - stay;
  int seen = before;
  for (int i0 = lo; i0 < hi; i0 += kStep) {
    int f = 0, n;
    const int i = i0 + p.tid * 4;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (i + e < hi && a.refs_in[i + e] != 0) f |= 1 << e;
    int k = seen + block_scan(__popc(f), sh, &n);  // used pages in front of page i
    seen += n;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int page = i + e;
      if (page >= hi) break;
      const bool on = f >> e & 1;
      a.remap[page] = on ? page : -1;
      if (on && page >= used) a.pairs[k - stay].x = page;
      if (!on && page < used) a.pairs[page - k].y = page;
      k += on;
    }
  }
  cluster_sync();  // the counts have been read: they may be moved where they lie
  copy_refs(a.refs_in, a.refs_out, a.num_pages, p);
  if (a.refs_in != a.refs_out) cluster_sync();
  for (int k = p.all; k < moves; k += p.n) {
    const int2 m = __ldcg(a.pairs + k);
    a.remap[m.x] = m.y;
    a.refs_out[m.y] = __ldcg(a.refs_out + m.x);
    a.refs_out[m.x] = 0;
  }
  if (p.all == 0) {
    *a.n_pairs = moves;
    *a.used = used;
  }
  cluster_sync();
  for (long long i = p.all; i < a.n; i += p.n) {
    const int page = a.pages_in[i];
    int to = -1;
    if (page >= 0 && page < a.num_pages) to = __ldcg(a.remap + page);
    if (to < 0 && page != -1) flag_error(a.err, kErrBadIndex);
    a.pages_out[i] = to;
  }
}

// ---- small pools: one CTA, counts and tables' sizes in shared memory -----------------------------------------------
// At most kFastPages pages and kFastRows requests and children: what the phases above exchange through L2 stays in the
// CTA, so that a call waits for memory two or three times (a fork of 32 samples of 61 blocks 14.3 -> 8.2 us, a step of
// 16 beams 12.8 -> 8.2, a page for each of 16 requests 6.2 -> 4.1, compaction's plan of 509 pages 10.3 -> 4.6; an empty
// launch takes 4.1).
constexpr int kFast = 512, kFastPer = 8, kFastPages = kFast * kFastPer, kFastRows = 512;

// Exclusive sums of two numbers over the CTA's kFast threads, and their totals. `sh`: 2 x 17 ints.
__device__ __forceinline__ int2 fast_scan(int2 x, int (*sh)[17], int2* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int2 v = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(kFull, v.x, o), b = __shfl_up_sync(kFull, v.y, o);
    if (lane >= o) v.x += a, v.y += b;
  }
  __syncthreads();
  if (lane == 31) sh[0][w] = v.x, sh[1][w] = v.y;
  __syncthreads();
  int2 before = make_int2(0, 0);
  *total = before;
#pragma unroll
  for (int i = 0; i < kFast / 32; ++i) {
    const int a = sh[0][i], b = sh[1][i];
    if (i < w) before.x += a, before.y += b;
    total->x += a;
    total->y += b;
  }
  return make_int2(before.x + v.x - x.x, before.y + v.y - x.y);
}
// The thread's kFastPer pages from tid * kFastPer on: its bits of those that are free (past the pool: none).
template <typename F>
__device__ __forceinline__ int own_pages(int pages, F is) {
  int m = 0;
#pragma unroll
  for (int e = 0; e < kFastPer; ++e) {
    const int page = threadIdx.x * kFastPer + e;
    if (page < pages && is(page)) m |= 1 << e;
  }
  return m;
}

__global__ void __launch_bounds__(kFast) pages_alloc_fast_kernel(const int* refs_in, int* refs_out, int pages,
                                                                 const int* want, int n, int* out, int* err) {
  __shared__ int sh[2][17], s_page[kFastRows];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  int count[kFastPer];
#pragma unroll
  for (int e = 0; e < kFastPer; ++e) {
    const int page = tid * kFastPer + e;
    count[e] = page < pages ? refs_in[page] : 1;
  }
  const bool takes = tid < n && (!want || want[tid] != 0);
  int free = 0;
#pragma unroll
  for (int e = 0; e < kFastPer; ++e) free |= (count[e] == 0) << e;
  int2 total;
  const int2 at = fast_scan(make_int2(__popc(free), takes), sh, &total);
  int k = at.x;
#pragma unroll
  for (int e = 0; e < kFastPer; ++e) {
    const int page = tid * kFastPer + e;
    const bool take = (free >> e & 1) && k < total.y;
    if (take) s_page[k] = page;
    k += free >> e & 1;
    if (page < pages && (take || refs_in != refs_out)) refs_out[page] = take ? 1 : count[e];
  }
  __syncthreads();
  if (tid < n) out[tid] = takes && at.y < total.x ? s_page[at.y] : -1;
  if (tid == 0 && total.y > total.x) flag_error(err, kErrNoPages);
}

__global__ void __launch_bounds__(kFast) pages_fork_fast_kernel(const ForkArgs a) {
  __shared__ int sh[2][17];
  __shared__ int s_refs[kFastPages];
  __shared__ Parent s_par[kFastRows];
  __shared__ int s_kids[kFastRows], s_first[kFastRows];
  // a child's parent and first entry; a copy's entry
  __shared__ int s_of[kFastRows], s_to[kFastRows + 1], s_at[kFastRows];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, wid = tid >> 5;
  for (int p = tid; p < a.num_pages; p += kFast) s_refs[p] = a.refs_in[p];
  if (tid < a.bt.R) {
    s_par[tid] = parent_of(a, tid);
    s_kids[tid] = 0;
    s_first[tid] = INT_MAX;
  }
  const int r = tid < a.F ? a.parent[tid] : -1;
  __syncthreads();
  const bool ok = tid < a.F && r >= 0 && r < a.bt.R && s_par[r].n >= 0;
  if (ok) {
    atomicAdd(s_kids + r, 1);
    atomicMin(s_first + r, tid);
  } else if (tid < a.F) {
    flag_error(a.err, kErrBadIndex);
  }
  __syncthreads();
  const int n = ok ? s_par[r].n : 0;
  const bool copy = ok && s_par[r].part && (a.keep || s_first[r] != tid);
  int2 total;
  const int2 at = fast_scan(make_int2(n, copy), sh, &total);
  if (tid < a.F) {
    s_of[tid] = n ? r : -1;
    s_to[tid] = at.x;
    a.child_offsets[tid] = at.x;
    a.child_lens[tid] = ok ? s_par[r].T : 0;
    if (copy) {
      s_at[at.y] = at.x + n - 1;
      a.pairs[at.y].x = a.bt.pages[s_par[r].off + n - 1];
    }
  }
  if (tid == 0) s_to[a.F] = a.child_offsets[a.F] = total.x;
  __syncthreads();
  bool missing = false;
  auto places = [&](auto f) {  // as above
    share_warps(wid, kFast / 32, a.bt.R, [&](int q, int j0, int step) {
      const Parent x = s_par[q];
      const int kids = s_kids[q];
      if (x.n < 0 && !a.keep && j0 == 0) flag_error(a.err, kErrBadIndex);
      for (int j = j0; j < x.n; j += step) {
        const int page = a.bt.pages[x.off + j];
        if (page < 0 || page >= a.num_pages) flag_error(a.err, kErrBadIndex);
        else f(page, change_of(a, kids, j == x.n - 1 && x.part));
      }
    });
  };
  places([&](int page, int more) {
    if ((more ? atomicAdd(s_refs + page, more) : s_refs[page]) <= 0) missing = true;
  });
  share_warps(wid, kFast / 32, a.F, [&](int i, int j0, int step) {
    const int q = s_of[i];
    if (q < 0) return;
    const Parent x = s_par[q];
    const int own = x.part && (a.keep || s_first[q] != i);  // the last entry is the copy's
    for (int j = j0; j < x.n - own; j += step) a.child_pages[s_to[i] + j] = a.bt.pages[x.off + j];
  });
  if (__syncthreads_or(missing)) {
    if (tid == 0) flag_error(a.err, kErrBadIndex);
    places([&](int page, int more) { atomicSub(s_refs + page, more); });
    __syncthreads();
    places([&](int page, int more) { make_count(s_refs + page, more); });
    __syncthreads();
    for (int p = tid; p < a.num_pages; p += kFast) s_refs[p] = real_count(s_refs[p]);
    __syncthreads();
  }
  const int free = own_pages(a.num_pages, [&](int page) { return s_refs[page] == 0; });
  const int need = total.y;
  int2 found;
  int k = fast_scan(make_int2(__popc(free), 0), sh, &found).x;
#pragma unroll
  for (int e = 0; e < kFastPer; ++e)
    if (free >> e & 1) {
      if (k < need) {
        const int page = tid * kFastPer + e;
        s_refs[page] = 1;
        a.pairs[k].y = page;
        a.child_pages[s_at[k]] = page;
      }
      ++k;
    }
  for (k = found.x + tid; k < need; k += kFast) a.child_pages[s_at[k]] = -1;
  __syncthreads();
  for (int p = tid; p < a.num_pages; p += kFast) a.refs_out[p] = s_refs[p];
  if (tid == 0) {
    *a.n_pairs = min(found.x, need);
    if (found.x < need) flag_error(a.err, kErrNoPages);
  }
}

__global__ void __launch_bounds__(kFast) pages_compact_fast_kernel(const CompactArgs a) {
  __shared__ int sh[2][17], s_stay;
  __shared__ int s_refs[kFastPages], s_map[kFastPages];
  __shared__ unsigned short s_from[kFastPages / 2], s_to[kFastPages / 2];
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x;
  for (int p = tid; p < a.num_pages; p += kFast) s_refs[p] = a.refs_in[p];
  __syncthreads();
  const int on = own_pages(a.num_pages, [&](int page) { return s_refs[page] != 0; });
  int2 total;
  const int first = fast_scan(make_int2(__popc(on), 0), sh, &total).x;
  const int used = total.x;
  // used pages in front of page `used`
  if (used / kFastPer == tid) s_stay = first + __popc(on & ((1 << used % kFastPer) - 1));
  if (tid == 0 && used == kFastPages) s_stay = used;
  __syncthreads();
  const int stay = s_stay, moves = used - stay;
  int k = first;
#pragma unroll
  for (int e = 0; e < kFastPer; ++e) {
    const int page = tid * kFastPer + e;
    if (page >= a.num_pages) break;
    const bool in = on >> e & 1;
    s_map[page] = in ? page : -1;
    if (in && page >= used) s_from[k - stay] = (unsigned short)page;
    if (!in && page < used) s_to[page - k] = (unsigned short)page;
    k += in;
  }
  __syncthreads();
  for (int i = tid; i < moves; i += kFast) {
    const int from = s_from[i], to = s_to[i];
    a.pairs[i] = make_int2(from, to);
    s_map[from] = to;
    s_refs[to] = s_refs[from];
    s_refs[from] = 0;
  }
  if (tid == 0) {
    *a.n_pairs = moves;
    *a.used = used;
  }
  __syncthreads();
  for (int p = tid; p < a.num_pages; p += kFast) {
    a.remap[p] = s_map[p];
    a.refs_out[p] = s_refs[p];
  }
  for (long long i = tid; i < a.n; i += kFast) {
    const int page = a.pages_in[i];
    const int to = page >= 0 && page < a.num_pages ? s_map[page] : -1;
    if (to < 0 && page != -1) flag_error(a.err, kErrBadIndex);
    a.pages_out[i] = to;
  }
}

// One page of an array is a run of vectors, slice after slice, cut into chunks of kUnroll a thread (a chunk spans
// slices where they are small); CTAs take (pair, chunk) in turn.
constexpr int kCopy = 256, kUnroll = 8, kChunk = kCopy * kUnroll;

template <typename V>
__device__ __forceinline__ void copy_chunk(const PageArray& d, const int2 m, int first) {
  if (d.whole) {  // the chunk is a run of one slice
    const int s = first / d.per;
    const long long at = s * d.slice + (long long)(first - s * d.per + (int)threadIdx.x) * (int)sizeof(V);
    const V* from = reinterpret_cast<const V*>(d.base + m.x * d.page + at);
    V* to = reinterpret_cast<V*>(d.base + m.y * d.page + at);
    V x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) x[u] = __ldcs(from + u * kCopy);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) to[u * kCopy] = x[u];
    return;
  }
  const int left = d.vecs - first - (int)threadIdx.x;  // vectors of the page from the thread's first on
  const int s0 = (first + (int)threadIdx.x) / d.per, o0 = first + (int)threadIdx.x - s0 * d.per;
  V x[kUnroll];
  // from one of a thread's vectors to the next: `step` bytes, or `step` and on to the next slice
  const long long step = d.step_s * d.slice + d.step_o * (int)sizeof(V);
  const long long over = d.slice - (long long)d.per * (int)sizeof(V);
  auto each = [&](auto f) {
    long long at = s0 * d.slice + (long long)o0 * (int)sizeof(V);
    int o = o0;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (u * kCopy < left) f(u, at);
      at += step;
      o += d.step_o;
      if (o >= d.per) o -= d.per, at += over;
    }
  };
  const char* from = d.base + m.x * d.page;
  each([&](int u, long long at) { x[u] = __ldcs(reinterpret_cast<const V*>(from + at)); });
  char* to = d.base + m.y * d.page;
  each([&](int u, long long at) { *reinterpret_cast<V*>(to + at) = x[u]; });
}

__global__ void __launch_bounds__(kCopy, 3) pages_copy_kernel(const __grid_constant__ PageArrays pa,
                                                              const int2* pairs, const int* n_pairs, int num_pages) {
  pdl_wait();
  pdl_launch_dependents();
  const long long units = (long long)*n_pairs * pa.chunks;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long pair = udiv(u, pa.chunks);
    const int c = (int)(u - pair * pa.chunks);
    const int2 m = pairs[pair];
    if (m.x < 0 || m.x >= num_pages || m.y < 0 || m.y >= num_pages) continue;  // a bad page of a parent's table
    int x = 0;
    while (x + 1 < pa.n && c >= pa.a[x + 1].first) ++x;
    const PageArray& d = pa.a[x];
    if (d.vec == 16) copy_chunk<uint4>(d, m, (c - d.first) * kChunk);
    else copy_chunk<uint32_t>(d, m, (c - d.first) * kChunk);
  }
}

// A planning kernel, which may start while the launch before it ends.
template <typename... P, typename... A>
cudaError_t launch_cluster(void (*k)(P...), int ctas, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

// The planning cluster: as many CTAs as there is work for.
template <typename... P, typename... A>
cudaError_t launch_plan(void (*k)(P...), long long work, cudaStream_t s, A... args) {
  int ctas = 1;
  while (ctas < kPlanCtas && work > (long long)ctas * kStep) ctas *= 2;
  return launch_cluster(k, ctas, kPlan, s, args...);
}
cudaError_t launch_copies(const PageArrays& pa, const int2* pairs, const int* n_pairs, long long most, int num_pages,
                          cudaStream_t s) {
  if (pa.n == 0 || most == 0) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::max(1ll, std::min(most * pa.chunks, 8ll * sm_count())));
  cfg.blockDim = dim3(kCopy);
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pages_copy_kernel, pa, pairs, n_pairs, num_pages);
}

}  // namespace

bool plan_page_arrays(PageArrays* pa) {
  pa->chunks = 0;
  for (int i = 0; i < pa->n; ++i) {
    PageArray& d = pa->a[i];
    const uintptr_t all = reinterpret_cast<uintptr_t>(d.base) | d.slice | d.page | d.bytes;
    d.vec = all % 16 ? 4 : 16;
    const long long per = d.bytes / d.vec, vecs = per * d.slices, chunks = (vecs + kChunk - 1) / kChunk;
    if (per > 0x7FFF0000 || vecs > 0x7FFF0000 || pa->chunks + chunks > 0x7FFF0000) return false;
    d.per = (int)per;
    d.vecs = (int)vecs;
    d.step_s = kCopy / d.per;
    d.step_o = kCopy % d.per;
    d.whole = d.per % kChunk == 0;
    d.first = pa->chunks;
    pa->chunks += (int)chunks;
  }
  return true;
}

cudaError_t launch_pages_alloc(const int* refs_in, int* refs_out, int num_pages, const int* want, int n, int* out,
                               int* err, cudaStream_t s) {
  if (num_pages <= kFastPages && n <= kFastRows)
    return launch_cluster(pages_alloc_fast_kernel, 1, kFast, s, refs_in, refs_out, num_pages, want, n, out, err);
  return launch_plan(pages_alloc_kernel, num_pages, s, refs_in, refs_out, num_pages, want, n, out, err);
}

cudaError_t launch_pages_free(const Table& bt, const int* refs_in, int* refs_out, int num_pages, int* err,
                              cudaStream_t s) {
  const long long work = (long long)bt.R * bt.max_blocks + (refs_in == refs_out ? 0 : num_pages);
  return launch_plan(pages_free_kernel, work, s, bt, refs_in, refs_out, num_pages, err);
}

cudaError_t launch_pages_fork(const ForkArgs& f, const PageArrays& pa, cudaStream_t s) {
  const long long work = std::max<long long>(f.num_pages, 2ll * f.F * f.bt.max_blocks);
  const bool fast = f.num_pages <= kFastPages && f.F <= kFastRows && f.bt.R <= kFastRows && work <= 4 * kStep;
  const cudaError_t e =
      fast ? launch_cluster(pages_fork_fast_kernel, 1, kFast, s, f) : launch_plan(pages_fork_kernel, work, s, f);
  return e != cudaSuccess ? e : launch_copies(pa, f.pairs, f.n_pairs, f.F, f.num_pages, s);
}

cudaError_t launch_pages_compact(const CompactArgs& c, const PageArrays& pa, cudaStream_t s) {
  const bool fast = c.num_pages <= kFastPages && c.n <= 4 * kStep;
  const cudaError_t e = fast ? launch_cluster(pages_compact_fast_kernel, 1, kFast, s, c)
                             : launch_plan(pages_compact_kernel, std::max<long long>(c.num_pages, c.n / 2), s, c);
  return e != cudaSuccess ? e : launch_copies(pa, c.pairs, c.n_pairs, c.num_pages / 2, c.num_pages, s);
}

}  // namespace kk
