// Offsets, block tables and slots of a ragged step from its request lengths
// (gdn_slot_map).
//
// Two prefix sums over the requests (new tokens, needed blocks), then one entry
// for each token and each needed block. Bound by latency for a few requests and
// by the 16 bytes a token of its outputs for many. One launch: every CTA scans
// all requests (a few KB, from L2), 1024 at a time with carried sums, and fills
// its own tokens and blocks of each batch of 1024 by bisection in shared memory;
// no CTA waits for another. With tokens enough a thread fills four in a row, in 16-byte
// stores, and looks for the request of the first only; positions of a good request are
// below 2^31, so the divisions by the block size are 32-bit ones. In a graph 8 requests
// take 3.5 us and 524289 tokens of 2048 requests 11.4, of which the bytes are 1.3: the rest
// is the two batches' chain of loads, scans and barriers (a batch is a request a thread, the
// second starts where the first has ended, and every CTA goes through both).
#include "gdn_prefill.cuh"

namespace gdn {
namespace {

constexpr int kSlotThreads = 1024;

struct Tile {
  long long tok[kSlotThreads + 1];   // first token of each request, and the end
  long long need[kSlotThreads + 1];  // blocks needed before each request
  int ctx[kSlotThreads];
  int have[kSlotThreads];            // blocks held; -1: the request gets none
  long long warp_tok[32], warp_need[32];
};

__device__ __forceinline__ long long warp_scan(long long v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Last i in [0, n) with a[i] <= v (a[0] <= v, a not decreasing).
__device__ __forceinline__ int last_at_most(const long long* a, int n, long long v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= v)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kSlotThreads) slot_map_kernel(const SlotParams p) {
  __shared__ Tile t;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first_cta = blockIdx.x == 0;
  const long long B = p.B;
  const int avail = min(max(*p.free_count, 0), p.free_cap);
  // this CTA's tokens
  const long long per = (((long long)p.N + gridDim.x - 1) / gridDim.x + 3) & ~3LL;
  const bool wide = ((reinterpret_cast<uintptr_t>(p.token_seq) | reinterpret_cast<uintptr_t>(p.token_pos) |
                      reinterpret_cast<uintptr_t>(p.slots)) & 15) == 0;
  const long long my0 = min((long long)p.N, per * blockIdx.x), my1 = min((long long)p.N, my0 + per);
  long long tok_carry = 0, need_carry = 0;
  long long taken = 0;
  for (long long at_request = 0; at_request < p.R; at_request += kSlotThreads) {
    const int base = (int)at_request, n = min(kSlotThreads, p.R - base), r = base + tid;
    long long nl = 0, cl = 0, have = 0, need = 0;
    bool bad = false;
    if (tid < n) {
      const int a = __ldg(p.new_lens + r), c = __ldg(p.ctx_lens + r);
      nl = max(a, 0);
      cl = max(c, 0);
      // rounded up: the sums are below 2^32
      const unsigned end = (unsigned)min(cl + nl, 0x7fffffffLL);
      have = ((unsigned)cl + (unsigned)p.B - 1) / (unsigned)p.B;
      const long long want = (end + (unsigned)p.B - 1) / (unsigned)p.B;
      bad = a < 0 || c < 0 || want > p.max_blocks || cl + nl > 0x7fffffffLL;
      need = bad ? 0 : want - have;
    }
    long long tok = warp_scan(nl), blk = warp_scan(need);
    if (lane == 31) {
      t.warp_tok[warp] = tok;
      t.warp_need[warp] = blk;
    }
    __syncthreads();
    if (warp == 0) {
      const long long a = warp_scan(t.warp_tok[lane]), b = warp_scan(t.warp_need[lane]);
      t.warp_tok[lane] = a;
      t.warp_need[lane] = b;
    }
    __syncthreads();
    if (warp) {
      tok += t.warp_tok[warp - 1];
      blk += t.warp_need[warp - 1];
    }
    tok += tok_carry;  // inclusive sums
    blk += need_carry;
    const bool fits = need == 0 || blk <= avail;
    t.tok[tid + 1] = tok;
    t.need[tid + 1] = blk;
    if (tid == 0) {
      t.tok[0] = tok_carry;
      t.need[0] = need_carry;
    }
    t.ctx[tid] = (int)cl;
    t.have[tid] = bad || !fits ? -1 : (int)have;
    if (first_cta && tid < n) {
      p.cu[r] = (int)min(tok - nl, (long long)p.N);
      if (bad && p.error) record(p.error, kStatusIndex, 1, r);
      if (!fits && p.error) record(p.error, kStatusIndex, 2, r);
    }
    __syncthreads();
    tok_carry = t.tok[kSlotThreads];
    need_carry = t.need[kSlotThreads];
    // the sums do not decrease, so what fits is a prefix of them
    if (need_carry <= avail)
      taken = need_carry;
    else if (t.need[0] <= avail)
      taken = t.need[last_at_most(t.need, kSlotThreads + 1, avail)];
    // tokens of this batch that are this CTA's
    const long long a0 = max(my0, t.tok[0]), a1 = min(my1, tok_carry);
    const auto entry = [&](int i, long long k, int* at, long long* slot) {
      const long long pos = t.ctx[i] + (k - t.tok[i]);
      *at = (int)min(pos, 0x7fffffffLL);
      *slot = -1;
      if (t.have[i] < 0) return;
      // a block of this step comes off the free list; an older one is in the table
      const int col = (unsigned)*at / (unsigned)p.B;
      const long long block = col >= t.have[i] ? __ldg(p.free_list + (avail - 1 - (t.need[i] + col - t.have[i])))
                                               : p.table[(long long)(base + i) * p.max_blocks + col];
      *slot = block * B + (*at - (long long)col * B);
    };
    const auto single = [&](long long k) {
      const int i = last_at_most(t.tok, n, k);
      int at;
      long long slot;
      entry(i, k, &at, &slot);
      p.token_seq[k] = base + i;
      p.token_pos[k] = at;
      p.slots[k] = slot;
    };
    if (!wide || a1 - a0 <= kSlotThreads) {
      for (long long k = a0 + tid; k < a1; k += kSlotThreads) single(k);
    } else {
      const long long v0 = (a0 + 3) & ~3LL, v1 = a1 & ~3LL;
      if (tid < 3 && a0 + tid < v0) single(a0 + tid);
      if (tid < 3 && v1 + tid < a1) single(v1 + tid);
      for (long long k = v0 + 4 * tid; k < v1; k += 4 * kSlotThreads) {
        int seq[4], at[4];
        long long slot[4];
        int i = last_at_most(t.tok, n, k);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          while (t.tok[i + 1] <= k + j) ++i;  // the token is before the batch's end, so this ends
          seq[j] = base + i;
          entry(i, k + j, &at[j], &slot[j]);
        }
        *reinterpret_cast<int4*>(p.token_seq + k) = make_int4(seq[0], seq[1], seq[2], seq[3]);
        *reinterpret_cast<int4*>(p.token_pos + k) = make_int4(at[0], at[1], at[2], at[3]);
        *reinterpret_cast<longlong2*>(p.slots + k) = make_longlong2(slot[0], slot[1]);
        *reinterpret_cast<longlong2*>(p.slots + k + 2) = make_longlong2(slot[2], slot[3]);
      }
    }
    // an even share of the batch's needed blocks, of which there can be 2^31 - 1
    const unsigned blocks = (unsigned)max(0LL, min(need_carry, taken) - t.need[0]);
    const unsigned share = (blocks + gridDim.x - 1) / gridDim.x, b0 = share * blockIdx.x, b1 = min(blocks, b0 + share);
    for (unsigned u = b0 + tid; u < b1; u += kSlotThreads) {
      const long long k = t.need[0] + u;
      const int i = last_at_most(t.need, n, k);
      p.table[(long long)(base + i) * p.max_blocks + t.have[i] + (k - t.need[i])] = __ldg(p.free_list + (avail - 1 - k));
    }
    __syncthreads();
  }
  // tokens past the last request
  for (long long k = max(my0, tok_carry) + tid; k < my1; k += kSlotThreads) {
    p.token_seq[k] = -1;
    p.token_pos[k] = -1;
    p.slots[k] = -1;
  }
  if (first_cta && tid == 0) {
    p.cu[p.R] = (int)min(tok_carry, (long long)p.N);
    *p.free_count_out = avail - (int)taken;
    if (tok_carry > p.N && p.error) record(p.error, kStatusIndex, 3, 0);
  }
}

}  // namespace

cudaError_t launch_slot_map(const SlotParams& p, cudaStream_t s) {
  // a CTA for every 2048 tokens, one for each SM at most
  const int grid = min(152, max(1, (p.N - 1) / 2048 + 1));
  slot_map_kernel<<<grid, kSlotThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn
