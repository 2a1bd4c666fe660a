// Eviction from a paged cache (selection, then the move) and commitment of
// an accepted path: copies of whole key and value rows by 16-byte pieces.
#include "tree_common.cuh"

namespace sv {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelPer = 16;  // consecutive tokens per thread
constexpr int kSelHeld = kSelThreads * kSelPer;  // tokens whose keys stay in registers
// Keys whose ranks are taken.  32 / 96 / 256: a batch cut to 2000 tokens a head
// 60.2 / 60.2 / 61.7 us.
constexpr int kSelList = 96;

// A weight's order as an unsigned integer: larger is better, NaN the worst.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Of tokens [lo, hi) of a longer row, the key of the need-th largest and how
// many of its equals are kept: a radix select over the order keys (11, 11
// and 10 bits), reading the weights three times.
__device__ __noinline__ uint32_t select_long(const float* w, int lo, int hi, int* need_io) {
  __shared__ int hist[2048];
  __shared__ int warp_tot[kSelThreads / 32];
  __shared__ int pick[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int need = *need_io, shift = 32;
  uint32_t prefix = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10;
    const int above = shift;  // bits fixed: [above, 32)
    shift -= bits;
    for (int i = tid; i < 2048; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int j = lo + tid; j < hi; j += kSelThreads) {
      const uint32_t k = weight_key(w[j]);
      if (above == 32 || (k >> above) == (prefix >> above)) atomicAdd(&hist[(k >> shift) & ((1u << bits) - 1u)], 1);
    }
    __syncthreads();
    // bins from the top: thread t holds bins 2047 - 2t and 2046 - 2t
    const int x = hist[2047 - 2 * tid], y = hist[2046 - 2 * tid];
    int v = x + y;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    if (lane == 31) warp_tot[warp] = v;
    __syncthreads();
    int base = 0;
    for (int i = 0; i < warp; ++i) base += warp_tot[i];
    const int incl = base + v, excl = incl - x - y;
    if (excl < need && incl >= need) {  // one thread
      const bool first = excl + x >= need;
      pick[0] = first ? 2047 - 2 * tid : 2046 - 2 * tid;
      pick[1] = need - (first ? excl : excl + x);
    }
    __syncthreads();
    prefix |= (uint32_t)pick[0] << shift;
    need = pick[1];
    __syncthreads();
  }
  *need_io = need;
  return prefix;
}

// One CTA per (request, head): the key of the last kept token and how many of
// its equals are kept, then a pass in token order writes the kept positions.
//
// Rows of up to kSelHeld tokens are read once, their keys held in registers.
// A key's bits are found two by two, by counts of the whole CTA, until few
// keys are left between the bounds; these go to a list, where ranks decide.
// Barriers and comparisons bound it, not bytes: 16 requests of 8 heads and up to
// 16384 tokens, 128 CTAs, take 15 us for 5 MB.  Bit by bit, one request cut from
// 4000 tokens takes 14.4 us with its move, two by two 13.4 (on the device alone;
// 15 to 17 with what launches from the host add); of 16384 tokens both take as
// long.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams P) {
  __shared__ int counts[2][kSelThreads / 32];
  __shared__ uint32_t list[kSelList];
  __shared__ int n_list, picked[2];
  __shared__ unsigned long long warp_tot2[kSelThreads / 32];
  after_previous();
  const int h = blockIdx.x % P.heads, b = blockIdx.x / P.heads;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int len = P.len[b];
  bool ok = len >= 0 && len <= P.ld && (long long)len <= (long long)P.ld_table * P.page_size;
  const int m = ok ? min(len, P.keep) : 0;
  const float* w = P.weights + ((long long)b * P.heads + h) * P.ld;
  const bool held = len <= kSelHeld;
  const int lo = P.sink, hi = len - P.recent;  // chosen by weight: [lo, hi)
  float x[kSelPer];
#pragma unroll
  for (int e = 0; e < kSelPer; ++e) x[e] = 0.f;
  if (ok && held) {
    // by 16 bytes where rows start on 16 (a row's last vector may pass its
    // length, not ld); by 4 a warp's loads touch every sector four times
    if (((reinterpret_cast<uintptr_t>(P.weights) | ((uintptr_t)P.ld * 4)) & 15) == 0) {
#pragma unroll
      for (int e = 0; e < kSelPer; e += 4)
        if (tid * kSelPer + e < len) {
          const float4 v = *reinterpret_cast<const float4*>(w + tid * kSelPer + e);
          x[e] = v.x;
          x[e + 1] = v.y;
          x[e + 2] = v.z;
          x[e + 3] = v.w;
        }
    } else {
#pragma unroll
      for (int e = 0; e < kSelPer; ++e)
        if (tid * kSelPer + e < len) x[e] = w[tid * kSelPer + e];
    }
  }
  int bad = 0;
  if (ok) {
    // both tables' first entries at once: latency is what short rows cost
    const int32_t* from_row = P.table + (long long)b * P.ld_table;
    const int32_t* to_row = P.to + (long long)b * P.ld_to;
    const int nf = len > 0 ? (len - 1) / P.page_size + 1 : 0, nt = m > 0 ? (m - 1) / P.page_size + 1 : 0;
    const int f0 = tid < nf ? from_row[tid] : 0, t0 = tid < nt ? to_row[tid] : 0;
    bad = f0 < 0 || f0 >= P.num_pages || t0 < 0 || t0 >= P.num_pages;
    for (int p = tid + kSelThreads; p < nf; p += kSelThreads) bad |= from_row[p] < 0 || from_row[p] >= P.num_pages;
    for (int p = tid + kSelThreads; p < nt; p += kSelThreads) bad |= to_row[p] < 0 || to_row[p] >= P.num_pages;
  }
  bad = __syncthreads_or(bad);
  int32_t* index = P.index + ((long long)b * P.heads + h) * P.keep;
  float* kept = P.kept ? P.kept + ((long long)b * P.heads + h) * P.keep : nullptr;
  if (h == 0 && tid == 0 && P.status) P.status[b] = !ok ? kStatusBadLen : (bad ? kStatusBadPage : 0);
  ok = ok && !bad;
  for (int i = (ok ? m : 0) + tid; i < P.keep; i += kSelThreads) {
    index[i] = -1;
    if (kept) kept[i] = 0.f;
  }
  if (!ok) return;
  const bool all = len <= P.keep;
  const int chosen = P.keep - P.sink - P.recent;
  int need = chosen;     // of the tokens of key `prefix` (not for `all`)
  uint32_t prefix = 0;   // the last kept key
  bool from = false;     // all tokens of that key are kept, and all above it
  uint32_t key[kSelPer];
  if (held) {
#pragma unroll
    for (int e = 0; e < kSelPer; ++e) {
      const int j = tid * kSelPer + e;
      key[e] = j >= lo && j < hi ? weight_key(x[e]) : 0u;  // 0 is NaN's: never probed
    }
  }
  if (!all && chosen > 0 && held) {
    // `at` keys are at or above prefix, chosen <= at; `above` are at or above
    // prefix + 2^left, above < chosen
    int above = 0, at = hi - lo, buf = 0;
    const bool some = warp * 32 * kSelPer < len;  // this warp holds keys
    if (tid == 0) n_list = 0;
    int left = 32;  // low bits of the key not found yet
#pragma unroll 1
    while (left > 0 && at != chosen && at - above > kSelList) {
      left -= 2;
      const uint32_t p1 = prefix + (1u << left), p2 = prefix + (2u << left), p3 = prefix + (3u << left);
      int n = 0;  // three counts: a warp's are at most 512
      if (some) {
#pragma unroll
        for (int e = 0; e < kSelPer; ++e) {
          n += key[e] >= p1 ? 1 : 0;
          n += key[e] >= p2 ? 1 << 10 : 0;
          n += key[e] >= p3 ? 1 << 20 : 0;
        }
        n = __reduce_add_sync(0xffffffffu, n);
      }
      if (lane == 0) counts[buf][warp] = n;
      __syncthreads();
      n = counts[buf][lane];
      buf ^= 1;  // the other one was read before this barrier
      const int n12 = __reduce_add_sync(0xffffffffu, (n & 1023) | ((n & (1023 << 10)) << 6));
      const int n1 = n12 & 0xffff, n2 = n12 >> 16, n3 = __reduce_add_sync(0xffffffffu, n >> 20);
      if (n3 >= chosen) {
        prefix = p3;
        at = n3;
      } else if (n2 >= chosen) {
        prefix = p2;
        at = n2;
        above = n3;
      } else if (n1 >= chosen) {
        prefix = p1;
        at = n1;
        above = n2;
      } else {
        above = n1;
      }
    }
    if (at == chosen) {
      from = true;
    } else if (left == 0) {
      need = chosen - above;  // more equals of one key than the list holds
    } else {
      // keys from prefix to below prefix + 2^left, by rank
      const uint32_t span = left == 32 ? 0xffffffffu : (1u << left) - 1u;
      __syncthreads();
      if (some) {
#pragma unroll
        for (int e = 0; e < kSelPer; ++e) {
          const int j = tid * kSelPer + e;
          if (j >= lo && j < hi && key[e] >= prefix && key[e] - prefix <= span) list[atomicAdd(&n_list, 1)] = key[e];
        }
      }
      __syncthreads();
      const int n = n_list, of = chosen - above;  // the of-th largest of the list
      if (tid < n) {
        const uint32_t k = list[tid];
        int more = 0, same = 0;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
          more += list[i] > k;
          same += list[i] == k;
        }
        if (more < of && more + same >= of) {  // one key, by all its equals alike
          picked[0] = (int)k;
          picked[1] = of - more;
        }
      }
      __syncthreads();
      prefix = (uint32_t)picked[0];
      need = picked[1];
    }
  } else if (!all && chosen > 0) {
    prefix = select_long(w, lo, hi, &need);
  }
  unsigned long long done = 0;  // kept without ties, ties (32 bits each)
  for (int base = 0; base < len; base += kSelHeld) {
    const int j0 = base + tid * kSelPer;
    uint32_t sure = 0, tie = 0;
#pragma unroll
    for (int e = 0; e < kSelPer; ++e) {
      const int j = j0 + e;
      if (j < len) {
        if (all || j < lo || j >= hi) {
          sure |= 1u << e;
        } else if (chosen > 0) {
          if (!held) x[e] = w[j];
          const uint32_t k = held ? key[e] : weight_key(x[e]);
          if (k > prefix || (from && k == prefix)) sure |= 1u << e;
          if (!from && k == prefix) tie |= 1u << e;
        }
      }
    }
    unsigned long long v = ((unsigned long long)__popc(sure) << 32) | (unsigned)__popc(tie);
    const unsigned long long mine = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    if (lane == 31) warp_tot2[warp] = v;
    __syncthreads();
    unsigned long long before = lane < warp ? warp_tot2[lane] : 0ull, sum = warp_tot2[lane];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      before += __shfl_xor_sync(0xffffffffu, before, o);
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    const unsigned long long at = done + before + v - mine;
    done += sum;
    // of this thread's ties the first that are still needed
    const int nt = (int)(at & 0xffffffffu), room = max(0, need - nt);
    while (__popc(tie) > room) tie &= ~(0x80000000u >> __clz(tie));
    int to = (int)(at >> 32) + min(nt, need);
    for (uint32_t take = sure | tie; take; take &= take - 1, ++to) {
      const int j = j0 + __ffs(take) - 1;
      index[to] = j;
      if (kept) kept[to] = w[j];
    }
    __syncthreads();
  }
}

// The move: 16-byte pieces of key and value rows, one kept token of a head
// per `pieces` lanes.  Bytes bound it: 2000 kept tokens of 128 heads of 128
// channels, 262 MB read and written, 41 us, 6.4 TB/s.  Threads per CTA, here
// and for the path, 64 / 128 / 256 / 512: with the selection 82 / 59.0 / 59.9 /
// 61.9 us, 64 requests' paths 19.4 / 17.3 / 16.9 / 20.5.
//
// The new lengths are written here, where every head's selection has ended, as
// they may take the place of the lengths that it read.
constexpr int kMoveThreads = 256;

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams P, int blocks) {
  const int part = blockIdx.x % blocks, bh = blockIdx.x / blocks;
  const int h = bh % P.heads, b = bh / P.heads;
  after_previous();
  const int pieces = P.dim / 8, per = kMoveThreads / pieces;
  const int i = part * per + (int)threadIdx.x / pieces, ch = threadIdx.x % pieces;
  if (i >= P.keep || (int)threadIdx.x >= per * pieces) return;
  const int j = P.index[((long long)b * P.heads + h) * P.keep + i];
  const bool first = i == 0 && ch == 0 && h == 0;
  if (j < 0) {  // past the kept tokens, or of an empty or bad request
    if (first) P.new_len[b] = P.len[b] == 0 ? 0 : -1;
    return;
  }
  const PageDiv pd(P.page_size);
  int ps, ss, pt, st;
  pd.split(j, ps, ss);
  pd.split(i, pt, st);
  const long long from = (long long)P.table[(long long)b * P.ld_table + ps] * P.s_page + (long long)ss * P.s_slot +
                         (long long)h * P.s_head + ch * 8;
  const long long to = (long long)P.to[(long long)b * P.ld_to + pt] * P.s_page + (long long)st * P.s_slot +
                       (long long)h * P.s_head + ch * 8;
  const uint4 k = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.k) + from);
  const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.v) + from);
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.k) + to) = k;
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.v) + to) = v;
  if (first) P.new_len[b] = min(P.len[b], P.keep);
}

// One CTA per (request, layer): checks the request, then copies its path.
// Latency bounds it, lengths to table to rows: 64 requests' paths of up to 33
// nodes in 28 layers of 4 heads of 128 channels, 89 MB read and written, 16.9
// us, 5.3 TB/s; one request's path 5.4 us.
//
// New lengths that take the place of the old ones, which every layer reads, are
// written by a launch of their own: P.new_len is null here, and there P.layers
// is 0.
__global__ void __launch_bounds__(kMoveThreads) commit_kernel(const CommitParams P) {
  after_previous();
  const int b = blockIdx.x, layer = blockIdx.y, tid = threadIdx.x;
  const int cu = P.cu[b], n = P.cu[b + 1] - cu, m = P.path_len[b], ctx = P.ctx[b];
  bool ok = cu >= 0 && n >= 0 && (long long)cu + n <= P.total && m >= 0 && m <= P.ld_path && ctx >= 0 &&
            (long long)ctx + m <= (long long)P.ld_table * P.page_size;
  const PageDiv pd(P.page_size);
  const int32_t* path = P.path + (long long)b * P.ld_path;
  const int32_t* table = P.table + (long long)b * P.ld_table;
  int bad = 0;
  if (ok)
    for (int i = tid; i < m; i += kMoveThreads) {
      int page, slot;
      pd.split(ctx + i, page, slot);
      const int node = path[i], id = table[page];
      bad |= (node < 0 || node >= n ? 1 : 0) | (id < 0 || id >= P.num_pages ? 2 : 0);
    }
  bool bad_node = false, bad_page = false;
  if (__syncthreads_or(bad)) {
    bad_node = __syncthreads_or(bad & 1) != 0;
    bad_page = __syncthreads_or(bad & 2) != 0;
  }
  if (layer == 0 && tid == 0) {
    const int st = (!ok || bad_node ? kStatusBadLen : 0) | (bad_page ? kStatusBadPage : 0);
    if (P.status) P.status[b] = st;
    if (P.new_len) P.new_len[b] = st ? -1 : ctx + m;
  }
  if (!ok || bad_node || bad_page || layer >= P.layers) return;
  // four pieces of keys and of values a thread in flight
  const int pieces = P.dim / 8, per_tok = P.heads * pieces, all = m * per_tok;
  constexpr int U = 4;
  for (int x0 = tid; x0 < all; x0 += U * kMoveThreads) {
    long long to[U];
    uint4 k[U], v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = x0 + u * kMoveThreads;
      if (x >= all) continue;
      const int i = x / per_tok, y = x - i * per_tok, h = y / pieces, ch = y - h * pieces;
      int page, slot;
      pd.split(ctx + i, page, slot);
      const long long from = (long long)layer * P.sn_layer + (long long)(cu + path[i]) * P.sn_node +
                             (long long)h * P.sn_head + ch * 8;
      to[u] = (long long)layer * P.s_layer + (long long)table[page] * P.s_page + (long long)slot * P.s_slot +
              (long long)h * P.s_head + ch * 8;
      k[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.k_new) + from);
      v[u] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(P.v_new) + from);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (x0 + u * kMoveThreads >= all) continue;
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.k) + to[u]) = k[u];
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.v) + to[u]) = v[u];
    }
  }
}

}  // namespace

int launch_evict(const EvictParams& P, cudaStream_t s) {
  if (launch_kernel(evict_select_kernel, dim3(P.B * P.heads), kSelThreads, 0, s, P)) return -1;
  const int per = kMoveThreads / (P.dim / 8), blocks = (P.keep + per - 1) / per;
  return launch_kernel(evict_move_kernel, dim3((unsigned)((long long)P.B * P.heads * blocks)), kMoveThreads, 0, s, P, blocks);
}

int launch_commit(const CommitParams& P, cudaStream_t s) {
  CommitParams Q = P;
  const bool in_place = P.new_len == P.ctx && P.layers > 1;
  if (in_place) Q.new_len = nullptr;
  if (launch_kernel(commit_kernel, dim3(P.B, P.layers), kMoveThreads, 0, s, Q)) return -1;
  if (!in_place) return 0;
  Q.new_len = P.new_len;
  Q.layers = 0;
  return launch_kernel(commit_kernel, dim3(P.B), kMoveThreads, 0, s, Q);
}

}  // namespace sv
