// Expert kernel of the few-token layer for bf16: the selected experts' gate/up
// and down products on tcgen05, the weights streamed once.
//
// The products are taken transposed: the weights' columns are the MMA's 128 rows
// (A, read MN-major as they lie in memory), the expert's tokens its columns
// (B, 16 to 128 of them), so one token costs no 128-row padding and a weight
// element passes through shared memory once whatever the number of tokens.
// With T tokens an expert there are 2 T FLOP a weight byte - far below the
// tensor cores' rate up to T = 128 - so HBM bounds the kernel: 3 H F bf16
// weights of every used expert.
//
// A unit of work is 64 rows (k) of two 128-column weight tiles: gate and up of
// the same columns, or two neighbouring tiles of W2; 32 KB either way.  All units of
// a phase form one line (slot, tile, k) that is cut into tickets of equal length
// whatever the tiles' borders, so the blocks stream the same number of bytes
// however few experts are used.  A ticket's piece of a tile that is not the whole
// tile leaves fp32 partial sums: of gate and up, the piece that arrives last adds
// the pieces in order and applies SwiGLU; of the down product, the weighted sum
// over the experts adds them in order while it reads them.  No sum depends on the
// order in which blocks run.  Measured, a call among others: 8 tokens 4096/64/4/2048 (26 experts,
// 1.3 GB of weights) 195 to 216 us by the experts used, 6.2 to 6.7 TB/s over the whole call; 64 tokens
// 4096/8/2/14336 432 to 453 us; 1 token 2048/64/6/1408 (104 MB) 30 to 33 us, of which 16
// are the weights.
//
// The activations pass to the down product as two bf16 numbers, the rounded value
// and what the rounding left, and y is as exact as with fp32 activations (relative
// error 0.0017, its own rounding; 0.0024 without).  Up to kSplitTokens tokens a slot both
// are columns of the same MMAs (1 % at most); beyond, where those columns would pass the
// accumulators' 128, a second MMA adds the rests to the same sums, so that a token's
// precision does not depend on how many others share its expert.
//
// With a few tokens the time is a chain of latencies, and the hand-over between the
// phases the longest of them: written, fenced, counted, added up, written, fenced,
// flagged, fetched - 8 us of a 1-token call's 36 (2048/64/6/1408).  Up to kDirectTokens
// tokens the partial sums carry their own flag instead: the router kernel fills
// their buffers with a NaN that no sum has (kEmpty), readers poll the very words
// that they need, and five warps build the down product's token tiles from them.
// With more tokens those tiles would be rebuilt from partial sums more often than
// they are worth.
//
// One block an SM, tickets taken in order (decode.cuh says why that cannot
// deadlock).  Warp 0 takes tickets and streams weights, running up to the whole
// ring (about 200 KB) ahead: it asks for the down tiles while the activations they
// meet are still being computed.  Warp 1 brings the tokens' rows: TMA row gathers of
// x, or rows of the activations once their slot is complete.  Warps 2 and 3 issue
// the MMAs of one tile each, warps 4-7 read TMEM (two accumulator sets) and write.
#include <cuda.h>
#include <string.h>

#include "decode.cuh"

namespace moe {
namespace decode {
namespace {

using namespace umma;

constexpr int kThreads = 256;
constexpr int kBuilders = 5;                // direct variant: warp 1 and four more build token tiles
constexpr int kDirectThreads = 384;
constexpr int kKB = 64;                     // rows of a unit
constexpr int kABytes = 4 * 8192;           // four 64 x 64 weight boxes
constexpr int kMaxStages = 6;
constexpr int kRing = 8;                    // tickets in flight in a block
constexpr int kUpTickets = 2, kDownTickets = 4;    // a block, on long lines
constexpr int kSmemData = 210 * 1024;
constexpr int kSplitTokens = 64;
constexpr int kPartFloats = 2 * 128;        // a token's sums of one piece

struct Params {
  CUtensorMap tw1, tw3, tw2;   // [E][H][F], [E][F][H]: 64 x 64 boxes
  CUtensorMap tx;              // [N][H]: one-row boxes, gathered
  CUtensorMap tact;            // [2][N*K][F]: 8-row boxes
  Args a;
  float* part_up;              // [2 * tickets][2][N][128]: a ticket's first piece, its last
  float* part_down;
  int* tile_cnt;               // [slots][F / 128] pieces that have arrived, zeroed by the router
  RouteCut cut;
  // of the ring, [1] where a slot holds more than kSplitTokens tokens
  int stages[2];
  int b_bytes[2];              // of a stage: the most rows of 128 bytes that its tokens take
};

struct Ticket {
  bool up, stop;
  int t;
};
__device__ __forceinline__ Ticket read_ticket(int v, const Line& up, const Line& down) {
  Ticket k;
  k.up = v < up.tickets;
  k.t = k.up ? v : v - up.tickets;
  k.stop = !k.up && k.t >= down.tickets;
  return k;
}

__device__ __forceinline__ int round16(int v) { return (v + 15) & ~15; }
__device__ __forceinline__ int round8(int v) { return (v + 7) & ~7; }
// The down product's token tile: the rounded activations from row 0 on, what the
// rounding left of them from row down_half(cnt) on; one_mma: columns of one MMA.
__device__ __forceinline__ bool one_mma(int cnt) { return cnt <= kSplitTokens; }
__device__ __forceinline__ int down_half(int cnt) { return one_mma(cnt) ? round8(cnt) : round16(cnt); }
// What rounding v to bf16 leaves; nothing of a value that is not finite as bf16.
__device__ __forceinline__ float rest_of(float v) {
  const float r = v - __bfloat162float(__float2bfloat16_rn(v));
  return isfinite(r) ? r : 0.f;
}
__device__ __forceinline__ uint32_t rest_of2(float a, float b) { return pack_bf16x2(rest_of(a), rest_of(b)); }
__device__ __forceinline__ void fence_proxy_async_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }
__device__ __forceinline__ void epi_barrier() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// All of the epilogue's threads: whether each of them says yes.  Its warps leave
// together or not at all, since they meet at barriers.
__device__ __forceinline__ bool epi_all(bool yes) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, 128, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((int)yes)
      : "memory");
  return r != 0;
}

// A warp after its lane 0 has waited: what lane 0 has seen is ordered before what the other lanes go on
// to write or copy (a shuffle alone orders no memory).
__device__ __forceinline__ bool lane0_says(bool ok) {
  __syncwarp();
  return __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
}

struct Shared {
  Plan plan;
  int tokens[kMaxTokens];      // warp 1's current slot
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[2], tempty[2];
  uint64_t ring_full[kRing], ring_empty[kRing];
  uint64_t drain[2];
  int ring[kRing];
  uint32_t tmem;
  int abort;
  int last;
  int ok;
  float4 sum[kThreads];
  Picked pick;
  // of the one or two tokens whose columns this block adds up
  float w[2][32];
  int row[2][32], tile[2][32], row0[2][32];
};
static_assert(kThreads == kRouteThreads, "pick_experts");

// Thread i of 2 K: expert i % K of the share's token i / K.
__device__ __forceinline__ void prepare_sum(const Args& a, Shared& sm, const Line& down, bool here, int i) {
  const Share h = share_of(a, kBlocks);
  const int ti = i / a.K, k = i - ti * a.K, n = h.first + ti;
  if (h.v0 >= h.v1 || n >= a.N) return;
  const int e = here ? sm.pick.id[n][k] : __ldcg(a.top + n * a.K + k);
  const int u = sm.plan.slot_of[e];
  sm.w[ti][k] = here ? sm.pick.w[n][k] : __ldcg(a.weights + n * a.K + k);
  sm.row[ti][k] = plan_row(sm.plan, n, e);
  sm.row0[ti][k] = sm.plan.off[u];
  sm.tile[ti][k] = u * down.nj;
}

// y[n] = sum_k w[n,k] out[row(n,k)], each out from its pieces in order.  Every
// block takes its share of the columns; nothing waits for it.  What does not
// depend on the down product is ready before the wait.  KL threads share the
// experts of four columns (thread kl those with k % KL = kl) and are added in
// order, KL as large as the share leaves threads for: with few columns a block the
// time is one chain of loads.
template <bool DIRECT>
__device__ __forceinline__ void weighted_sums(const Params& p, Shared& sm, const Line& down) {
  const Args& a = p.a;
  const int tid = threadIdx.x;
  const Share sh = share_of(a, kBlocks);
  const int per_row = sh.per_row, v0 = sh.v0, v1 = sh.v1, share = v1 - v0, first = sh.first;
  if (v0 >= v1) return;
  int KL = 1;
  while (KL < 8 && KL < a.K && 2 * KL * share <= kThreads) KL *= 2;
  const int VL = kThreads / KL, vl = tid % VL, kl = tid / VL;
  if (tid == 0) sm.ok = DIRECT || wait_count(&a.cnt->done_down, down.tickets, a.cnt, a.status);
  __syncthreads();
  if (!sm.ok) return;
  Patience patience;
  const size_t entry = (size_t)a.N * kPartFloats;
  for (int vb = v0; vb < v1; vb += VL) {
    const int at = vb + vl;
    const bool in = at < v1 && tid < kThreads;
    const int n = in ? at / per_row : first, h = in ? (at - n * per_row) * 4 : 0;
    const int ti = n - first, j = h >> 8;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (in) {
#pragma unroll 4
      for (int k = kl; k < a.K; k += KL) {
        const float w = sm.w[ti][k];
        const int row = sm.row[ti][k];
        const int a0 = (sm.tile[ti][k] + j) * down.kc;
        const int t0 = down.ticket_of(a0), t1 = down.ticket_of(a0 + down.kc - 1);
        const float* q0 = p.part_down + (size_t)((h >> 7) & 1) * a.N * 128 +
                          (size_t)(row - sm.row0[ti][k]) * 128 + (h & 127);
        const float* at0 = t0 == t1 ? a.out + (size_t)row * a.H + h : q0 + entry * down.entry(t0, a0);
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int t = t0; t <= t1; t += 4) {          // four pieces in flight
          float4 q[4];
          auto piece = [&](int i) { return t + i == t0 ? at0 : q0 + entry * (2 * (t + i)); };
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            q[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t + i <= t1) q[i] = DIRECT ? ld_words4(piece(i)) : __ldcg((const float4*)piece(i));
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (DIRECT)
              while (empty(q[i]) && patience.again(a.cnt, a.status)) q[i] = ld_words4(piece(i));
            o.x += q[i].x; o.y += q[i].y; o.z += q[i].z; o.w += q[i].w;
          }
        }
        s.x = fmaf(w, o.x, s.x); s.y = fmaf(w, o.y, s.y); s.z = fmaf(w, o.z, s.z); s.w = fmaf(w, o.w, s.w);
      }
    }
    if (KL > 1) {
      if (tid < kThreads) sm.sum[tid] = s;
      __syncthreads();
      if (kl == 0 && in) {
        for (int i = 1; i < KL; ++i) {
          const float4 q = sm.sum[i * VL + vl];
          s.x += q.x; s.y += q.y; s.z += q.z; s.w += q.w;
        }
      }
      __syncthreads();
    }
    if (kl == 0 && in)
      *(uint2*)((__nv_bfloat16*)a.y + (size_t)n * a.H + h) = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
  }
}

template <bool DIRECT>
__global__ void __launch_bounds__(DIRECT ? kDirectThreads : kThreads, 1)
decode_umma_kernel(const __grid_constant__ Params p) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ Shared sm;
  const Args& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  volatile int* abort_flag = &sm.abort;
  auto bar = [](const uint64_t& b) { return smem_u32(&b); };

  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(bar(sm.full[i]), 2);         // the weights' producer and the tokens'
      mbar_init(bar(sm.empty[i]), 2);        // both MMA warps
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(sm.tfull[i]), 2);
      mbar_init(bar(sm.tempty[i]), 4);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(bar(sm.ring_full[i]), 1);
      mbar_init(bar(sm.ring_empty[i]), 2 + 4 + (DIRECT ? kBuilders : 1));   // MMA, epilogue, tokens' rows
    }
    mbar_init(bar(sm.drain[0]), 1);
    mbar_init(bar(sm.drain[1]), 1);
    sm.abort = 0;
    fence_barrier_init();
  } else if (warp == 1 && lane < 5) {
    const CUtensorMap* m[5] = {&p.tw1, &p.tw3, &p.tw2, &p.tx, &p.tact};
    tma_prefetch_desc(m[lane]);
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&sm.tmem), 512);
    tmem_relinquish();
  }
  // tickets start at zero (the previous call's last block left them so), so the
  // first one can be taken while the router still runs
  int v = 0;
  if (tid == 0) v = atomicAdd(a.queue, 1);
  clear_plan(sm.plan, (int)blockDim.x);
  pdl_wait();
  if (p.cut.here) {
    float* red = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)));   // the ring is still empty
    pick_all(a, p.cut, sm.plan, sm.pick, red);
    build_plan(sm.plan, nullptr, a.N, a.K, a.E, (int)blockDim.x);
    fence_proxy_async();       // `red` was written where TMA will write
  } else {
    build_plan(sm.plan, a.top, a.N, a.K, a.E, (int)blockDim.x);
  }
  const int slots = sm.plan.slots;
  // Wider stages, and one fewer of them from 81 tokens on, only where a slot needs them: three stages
  // for every such call cost 3 % of those bound by HBM (128 tokens 4096/64/4/2048: 524 us with four,
  // 540 with three).  With all 128 tokens on one expert 4096/1/1/8192 the three and the second
  // MMAs cost 143 us against the 127 of activations rounded to one number.
  tc_fence_before();
  const int wide = __syncthreads_or(!DIRECT && tid < slots && !one_mma(sm.plan.off[tid + 1] - sm.plan.off[tid]));
  tc_fence_after();
  const int stages = p.stages[wide != 0];
  const uint32_t stage_bytes = kABytes + p.b_bytes[wide != 0];
  const uint32_t tmem = sm.tmem;
  // a quarter of the mean tokens a slot (60 tokens on each of two experts 2432/640: 77 us
  // without, 54 with), and eight units, so that short tiles stay whole (61 tokens
  // 256/6/4/1024: 38 us without, 30 with); four in the direct variant, where cuts cost less
  const int mean4 = (a.N * a.K / slots + 3) / 4, few = DIRECT ? 4 : 8, least = mean4 > few ? mean4 : few;
  const Line up = make_line(slots, a.F / 128, a.H / kKB, kUpTickets, least);
  const Line down = make_line(slots, (a.H + 255) / 256, a.F / kKB, kDownTickets, least);

  if (warp == (DIRECT ? kDirectThreads / 32 - 1 : 4))
    for (int i = lane; i < 2 * a.K; i += 32) prepare_sum(a, sm, down, p.cut.here, i);

  // the roles' view of the ticket ring
  int slot = 0;
  uint32_t ring_phase = 0;
  auto next_slot = [&]() {
    if (++slot == kRing) { slot = 0; ring_phase ^= 1u; }
  };

  if (warp == 0) {
    // ------------------------------------------------ tickets and weights
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (;;) {
      if (lane == 0) {
        ok = mbar_wait_bounded(bar(sm.ring_empty[slot]), ring_phase ^ 1u, abort_flag, a.status, kTimeoutNs);
        if (ok) {
          sm.ring[slot] = v;
          mbar_arrive(bar(sm.ring_full[slot]));
        }
      }
      ok = lane0_says(ok);
      if (!ok) break;
      const Ticket k = read_ticket(__shfl_sync(0xffffffffu, v, 0), up, down);
      if (k.stop) break;
      next_slot();
      {
        const Line& l = k.up ? up : down;
        const int begin = l.start(k.t), end = l.start(k.t + 1);
        for (int pos = begin; pos < end && ok;) {
          const Piece pc = piece_at(l, pos, end);
          const int u = pc.tile / l.nj, j = pc.tile - u * l.nj;
          const int e = sm.plan.expert[u];
          // lane 0-3: one 64-column box each
          const CUtensorMap* m = !k.up ? &p.tw2 : (lane < 2 ? &p.tw1 : &p.tw3);
          const int c = k.up ? j * 128 + (lane & 1) * 64 : j * 256 + lane * 64;
          for (int i = 0; i < pc.len; ++i) {
            if (lane == 0) {
              ok = mbar_wait_bounded(bar(sm.empty[stage]), phase ^ 1u, abort_flag, a.status, kTimeoutNs);
              if (ok) mbar_expect_tx(bar(sm.full[stage]), kABytes);
            }
            ok = lane0_says(ok);
            if (!ok) break;
            if (lane < 4)
              tma_load_3d(base + stage * stage_bytes + lane * 8192, m, bar(sm.full[stage]), c, (pc.k0 + i) * kKB, e);
            ++issued;
            if (++stage == stages) { stage = 0; phase ^= 1u; }
          }
          pos += pc.len;
        }
      }
      if (!ok) break;
      // not earlier: a block that runs ahead of the others would take work that
      // it can only queue, and the ring hides the round trip
      if (lane == 0) v = atomicAdd(a.queue, 1);
    }
    if (lane == 0) {
      // the copies in flight land before the block leaves, also after a wait gave up
      for (int i = 0; i < stages && i < issued; ++i) {
        if (stage-- == 0) { stage = stages - 1; phase ^= 1u; }
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(bar(sm.full[stage]), phase) && globaltimer() - t0 < 50000000ull) {}
      }
    }
  } else if (warp == 1 || (DIRECT && warp >= 8)) {
    // --------------------------------------------------------- the tokens' rows
    // (direct variant: the builders take a down ticket's units in turn)
    const int builder = warp == 1 ? 0 : warp - 7;
    const float* act32 = (const float*)a.act;
    const size_t entry = (size_t)a.N * kPartFloats;
    Patience patience;
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    int have = -1;                     // slot whose activations are known to be complete
    while (ok) {
      if (lane == 0) ok = mbar_wait_bounded(bar(sm.ring_full[slot]), ring_phase, abort_flag, a.status, kTimeoutNs);
      ok = lane0_says(ok);
      if (!ok) break;
      const Ticket k = read_ticket(*(volatile int*)&sm.ring[slot], up, down);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sm.ring_empty[slot]));
      next_slot();
      if (k.stop) break;
      const Line& l = k.up ? up : down;
      const int begin = l.start(k.t), end = l.start(k.t + 1);
      for (int pos = begin; pos < end && ok;) {
        const Piece pc = piece_at(l, pos, end);
        const int u = pc.tile / l.nj;
        const int e = sm.plan.expert[u], r0 = sm.plan.off[u], cnt = sm.plan.off[u + 1] - r0;
        const int rows = k.up ? round16(cnt) : 2 * down_half(cnt);
        int g0 = a.N, g1 = a.N, g2 = a.N, g3 = a.N;        // rows past the last token read as zeros
        if (DIRECT && k.up && builder != 0) {
          for (int i = 0; i < pc.len; ++i)
            if (++stage == stages) { stage = 0; phase ^= 1u; }
          pos += pc.len;
          continue;
        }
        if (k.up) {
          for (int n = lane; n < a.N; n += 32)
            if ((sm.plan.mask[e][n >> 5] >> (n & 31)) & 1u) sm.tokens[plan_row(sm.plan, n, e) - r0] = n;
          __syncwarp();
          if (4 * lane < cnt) g0 = sm.tokens[4 * lane];
          if (4 * lane + 1 < cnt) g1 = sm.tokens[4 * lane + 1];
          if (4 * lane + 2 < cnt) g2 = sm.tokens[4 * lane + 2];
          if (4 * lane + 3 < cnt) g3 = sm.tokens[4 * lane + 3];
          __syncwarp();
        } else if (!DIRECT && have != u) {
          if (lane == 0) {
            ok = wait_count(a.cnt->done_act + u, up.nj, a.cnt, a.status);
            if (!ok) *abort_flag = 1;
          }
          ok = lane0_says(ok);
          if (!ok) break;
          fence_proxy_async_global();                      // written by other threads, read by TMA
          have = u;
        }
        for (int i = 0; i < pc.len; ++i) {
          if (DIRECT && !k.up) {
            if ((pos + i) % kBuilders == builder) {
              // act[r][f] = silu(sum of gate pieces) * (sum of up pieces), lane: f = 2 lane, 2 lane + 1
              const int f = (pc.k0 + i) * kKB + 2 * lane;
              const int tile = u * up.nj + (f >> 7), a0 = tile * up.kc;
              const int t0 = up.ticket_of(a0), t1 = up.ticket_of(a0 + up.kc - 1);
              const float* first = p.part_up + entry * up.entry(t0, a0) + (f & 127);
              const float* rest = p.part_up + (f & 127);
              uint32_t v[kDirectTokens], lo[kDirectTokens];
#pragma unroll
              for (int r = 0; r < kDirectTokens; ++r) v[r] = lo[r] = 0u;
              if (t0 == t1) {
                float2 w[kDirectTokens];
                bool miss;
                do {
                  miss = false;
#pragma unroll
                  for (int r = 0; r < kDirectTokens; ++r)
                    if (r < cnt) w[r] = ld_words2(act32 + (size_t)(r0 + r) * a.F + f);
#pragma unroll
                  for (int r = 0; r < kDirectTokens; ++r)
                    if (r < cnt) miss |= empty(w[r]);
                } while (miss && patience.again(a.cnt, a.status));
#pragma unroll
                for (int r = 0; r < kDirectTokens; ++r)
                  if (r < cnt) {
                    v[r] = pack_bf16x2(w[r].x, w[r].y);
                    lo[r] = rest_of2(w[r].x, w[r].y);
                  }
              } else {
#pragma unroll
                for (int r = 0; r < kDirectTokens; ++r)
                  if (r < cnt) {
                    float2 g = make_float2(0.f, 0.f), w = g;
                    for (int t = t0; t <= t1; t += 4) {       // four pieces asked for at once
                      float2 gq[4], wq[4];
                      bool miss;
                      do {
                        miss = false;
#pragma unroll
                        for (int m = 0; m < 4; ++m) {
                          const float* q = (t + m == t0 ? first : rest + entry * (2 * (t + m))) + r * 128;
                          gq[m] = t + m <= t1 ? ld_words2(q) : make_float2(0.f, 0.f);
                          wq[m] = t + m <= t1 ? ld_words2(q + a.N * 128) : make_float2(0.f, 0.f);
                        }
#pragma unroll
                        for (int m = 0; m < 4; ++m) miss |= empty(gq[m]) || empty(wq[m]);
                      } while (miss && patience.again(a.cnt, a.status));
#pragma unroll
                      for (int m = 0; m < 4; ++m) {
                        g.x += gq[m].x; g.y += gq[m].y;
                        w.x += wq[m].x; w.y += wq[m].y;
                      }
                    }
                    const float ax = silu_f(g.x) * w.x, ay = silu_f(g.y) * w.y;
                    v[r] = pack_bf16x2(ax, ay);
                    lo[r] = rest_of2(ax, ay);
                  }
              }
              if (lane == 0) ok = mbar_wait_bounded(bar(sm.empty[stage]), phase ^ 1u, abort_flag, a.status, kTimeoutNs);
              ok = lane0_says(ok);
              if (!ok) break;
              const uint32_t dst = base + stage * stage_bytes + kABytes;
#pragma unroll
              for (int r = 0; r < kDirectTokens; ++r)      // 128-byte swizzle: 16-byte chunk ^ row
                if (r < cnt) {
                  const uint32_t at = dst + r * 128 + (((lane >> 2) ^ r) << 4) + (lane & 3) * 4;
                  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(v[r]) : "memory");
                  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + 1024), "r"(lo[r]) : "memory");   // row 8 + r
                }
              fence_proxy_async();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(sm.full[stage]));
            }
            if (++stage == stages) { stage = 0; phase ^= 1u; }
            continue;
          }
          if (lane == 0) {
            ok = mbar_wait_bounded(bar(sm.empty[stage]), phase ^ 1u, abort_flag, a.status, kTimeoutNs);
            if (ok) mbar_expect_tx(bar(sm.full[stage]), rows * 128);
          }
          ok = lane0_says(ok);
          if (!ok) break;
          const uint32_t dst = base + stage * stage_bytes + kABytes;
          const int kcol = (pc.k0 + i) * kKB;
          if (k.up) {
            if (4 * lane < rows) tma_gather4(dst + lane * 512, &p.tx, bar(sm.full[stage]), kcol, g0, g1, g2, g3);
          } else {
            // box b: rows 8 b on; the second half of the boxes are what the rounding left
            const int half = rows / 16;
            const int row = lane < half ? r0 + 8 * lane : a.N * a.K + r0 + 8 * (lane - half);
            if (8 * lane < rows) tma_load_2d(dst + lane * 1024, &p.tact, bar(sm.full[stage]), kcol, row);
          }
          ++issued;
          if (++stage == stages) { stage = 0; phase ^= 1u; }
        }
        pos += pc.len;
      }
    }
    if (lane == 0) {
      for (int i = 0; i < stages && i < issued; ++i) {
        if (stage-- == 0) { stage = stages - 1; phase ^= 1u; }
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(bar(sm.full[stage]), phase) && globaltimer() - t0 < 50000000ull) {}
      }
    }
  } else if (warp == 2 || warp == 3) {
    // --------------------------------------------------------------------- MMA
    // One thread takes some 75 cycles an MMA, about 800 a unit for both of its tiles,
    // and a ring that fills at once (activations that were waited for) empties no
    // faster: so a thread a tile.
    const int half = warp - 2;
    if (lane == 0) {
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      while (ok) {
        ok = mbar_wait_bounded(bar(sm.ring_full[slot]), ring_phase, abort_flag, a.status, kTimeoutNs);
        if (!ok) break;
        const Ticket k = read_ticket(*(volatile int*)&sm.ring[slot], up, down);
        mbar_arrive(bar(sm.ring_empty[slot]));
        next_slot();
        if (k.stop) break;
          const Line& l = k.up ? up : down;
        const int begin = l.start(k.t), end = l.start(k.t + 1);
        for (int pos = begin; pos < end && ok;) {
          const Piece pc = piece_at(l, pos, end);
          const int u = pc.tile / l.nj;
          const int cnt = sm.plan.off[u + 1] - sm.plan.off[u];
          const bool two = !DIRECT && !k.up && !one_mma(cnt);
          const uint32_t idesc = idesc_bf16(128, k.up || two ? round16(cnt) : 2 * down_half(cnt), true, false);
          ok = mbar_wait_bounded(bar(sm.tempty[acc]), acc_phase ^ 1u, abort_flag, a.status, kTimeoutNs);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem + acc * 256 + half * 128;
          for (int i = 0; i < pc.len; ++i) {
            ok = mbar_wait_bounded(bar(sm.full[stage]), phase, abort_flag, a.status, kTimeoutNs);
            if (!ok) break;
            tc_fence_after();
            const uint32_t sa = base + stage * stage_bytes + half * 16384, sb = base + stage * stage_bytes + kABytes;
#pragma unroll
            for (int kk = 0; kk < kKB / 16; ++kk)
              mma_bf16(d, desc_mn_sw128(sa + kk * 2048, 8192), desc_k_sw128(sb + kk * 32), idesc, (i | kk) != 0 ? 1u : 0u);
            if (two) {
              const uint32_t sr = sb + down_half(cnt) * 128;
#pragma unroll
              for (int kk = 0; kk < kKB / 16; ++kk)
                mma_bf16(d, desc_mn_sw128(sa + kk * 2048, 8192), desc_k_sw128(sr + kk * 32), idesc, 1u);
            }
            mma_commit(bar(sm.empty[stage]));
            if (++stage == stages) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          mma_commit(bar(sm.tfull[acc]));
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
          pos += pc.len;
        }
      }
      if (*abort_flag) {
        // the MMAs in flight still read shared memory and write TMEM
        mma_commit(bar(sm.drain[half]));
        const uint64_t t0 = globaltimer();
        while (!mbar_try_wait(bar(sm.drain[half]), 0) && globaltimer() - t0 < 50000000ull) {}
      }
    }
    __syncwarp();
  } else if (warp >= 4 && warp < 8) {
    // ---------------------------------------------------------------- epilogue
    const int et = tid - 128, quarter = warp & 3;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    __nv_bfloat16* act = (__nv_bfloat16*)a.act;
    const size_t act_rest = (size_t)a.N * a.K * a.F;
    auto put_act = [&](size_t at, float v) {
      act[at] = __float2bfloat16_rn(v);
      act[act_rest + at] = __float2bfloat16_rn(rest_of(v));
    };
    const size_t entry = (size_t)a.N * kPartFloats;        // floats of a partial-sum entry
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    while (ok) {
      if (lane == 0) ok = mbar_wait_bounded(bar(sm.ring_full[slot]), ring_phase, abort_flag, a.status, kTimeoutNs);
      ok = epi_all(ok);
      if (!ok) break;
      const Ticket k = read_ticket(*(volatile int*)&sm.ring[slot], up, down);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(sm.ring_empty[slot]));
      next_slot();
      if (k.stop) break;
      const Line& l = k.up ? up : down;
      const int begin = l.start(k.t), end = l.start(k.t + 1);
      for (int pos = begin; pos < end;) {
        const Piece pc = piece_at(l, pos, end);
        const int u = pc.tile / l.nj, j = pc.tile - u * l.nj;
        const int r0 = sm.plan.off[u], cnt = sm.plan.off[u + 1] - r0;
        const bool whole = pc.len == l.kc;
        if (lane == 0) ok = mbar_wait_bounded(bar(sm.tfull[acc]), acc_phase, abort_flag, a.status, kTimeoutNs);
        ok = epi_all(ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + acc * 256 + lanes;
        const int a0 = pc.tile * l.kc;
        float* part = (k.up ? p.part_up : p.part_down) + entry * l.entry(k.t, a0) + et;
        const int rest = !k.up && one_mma(cnt) ? down_half(cnt) : 0;    // columns from a value to its rest's
        for (int c = 0; c < cnt; c += 16) {
          uint32_t v0[16], v1[16];
          tmem_ld_16(d + c, v0);
          tmem_ld_16(d + 128 + c, v1);
          tmem_ld_wait();
          if (rest) {
            uint32_t l0[16], l1[16];
            tmem_ld_16(d + rest + c, l0);
            tmem_ld_16(d + 128 + rest + c, l1);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              v0[i] = __float_as_uint(__uint_as_float(v0[i]) + __uint_as_float(l0[i]));
              v1[i] = __float_as_uint(__uint_as_float(v1[i]) + __uint_as_float(l1[i]));
            }
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (c + i >= cnt) break;
            const float f0 = __uint_as_float(v0[i]), f1 = __uint_as_float(v1[i]);
            if (DIRECT) {
              const size_t row = r0 + c + i;
              if (!whole) {
                st_word(part + (c + i) * 128, f0);
                st_word(part + (a.N + c + i) * 128, f1);
              } else if (k.up) {
                st_word((float*)a.act + row * a.F + j * 128 + et, silu_f(f0) * f1);
              } else {
                float* o = a.out + row * a.H + j * 256 + et;
                st_word(o, f0);
                if (j * 256 + 128 < a.H) st_word(o + 128, f1);
              }
            } else if (!whole) {
              part[(c + i) * 128] = f0;
              part[((size_t)a.N + c + i) * 128] = f1;
            } else if (k.up) {
              put_act((size_t)(r0 + c + i) * a.F + j * 128 + et, silu_f(f0) * f1);
            } else {
              float* o = a.out + (size_t)(r0 + c + i) * a.H + j * 256 + et;
              o[0] = f0;
              if (j * 256 + 128 < a.H) o[128] = f1;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(sm.tempty[acc]));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1u;
        if (!DIRECT && k.up) {
          bool finish = whole;
          if (!whole) {
            // the last piece of the tile to arrive adds them all
            const int t0 = l.ticket_of(a0), t1 = l.ticket_of(a0 + l.kc - 1);
            epi_barrier();
            if (et == 0) {
              __threadfence();      // one thread's fence covers what the barrier has ordered before it
              sm.last = atomicAdd(p.tile_cnt + pc.tile, 1) == t1 - t0;
              __threadfence();
            }
            epi_barrier();
            finish = sm.last != 0;
            if (finish) {
              // a warp a token, four columns a lane; gate at q, up N * 128 floats on; three
              // pieces of four tokens in flight
              constexpr int PT = 3, TT = 4;
              const float* first = p.part_up + entry * l.entry(t0, a0) + lane * 4;
              const float* more = p.part_up + lane * 4;
              for (int c = quarter; c < cnt; c += 4 * TT) {
                float4 g[TT], w[TT];
#pragma unroll
                for (int r = 0; r < TT; ++r) g[r] = w[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int t = t0; t <= t1; t += PT) {
                  float4 gq[PT][TT], wq[PT][TT];
#pragma unroll
                  for (int i = 0; i < PT; ++i) {
                    const float* q = (t + i == t0 ? first : more + entry * (2 * (t + i))) + (size_t)c * 128;
#pragma unroll
                    for (int r = 0; r < TT; ++r) {
                      gq[i][r] = wq[i][r] = make_float4(0.f, 0.f, 0.f, 0.f);
                      if (t + i <= t1 && c + 4 * r < cnt) {
                        gq[i][r] = __ldcg((const float4*)(q + r * 512));
                        wq[i][r] = __ldcg((const float4*)(q + (size_t)a.N * 128 + r * 512));
                      }
                    }
                  }
#pragma unroll
                  for (int i = 0; i < PT; ++i)
#pragma unroll
                    for (int r = 0; r < TT; ++r) {
                      g[r].x += gq[i][r].x; g[r].y += gq[i][r].y; g[r].z += gq[i][r].z; g[r].w += gq[i][r].w;
                      w[r].x += wq[i][r].x; w[r].y += wq[i][r].y; w[r].z += wq[i][r].z; w[r].w += wq[i][r].w;
                    }
                }
#pragma unroll
                for (int r = 0; r < TT; ++r)
                  if (c + 4 * r < cnt) {
                    const float v0 = silu_f(g[r].x) * w[r].x, v1 = silu_f(g[r].y) * w[r].y;
                    const float v2 = silu_f(g[r].z) * w[r].z, v3 = silu_f(g[r].w) * w[r].w;
                    const size_t at = (size_t)(r0 + c + 4 * r) * a.F + j * 128 + lane * 4;
                    *(uint2*)(act + at) = make_uint2(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3));
                    *(uint2*)(act + act_rest + at) = make_uint2(rest_of2(v0, v1), rest_of2(v2, v3));
                  }
              }
            }
          }
          if (finish) {
            fence_proxy_async_global();
            epi_barrier();
            if (et == 0) add_release(a.cnt->done_act + u, 1);
          }
        }
        pos += pc.len;
      }
      if (!ok) break;
      if (!DIRECT && !k.up) {
        epi_barrier();
        if (et == 0) add_release(&a.cnt->done_down, 1);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 2) tmem_dealloc(tmem, 512);
  if (!sm.abort) weighted_sums<DIRECT>(p, sm, down);
  __syncthreads();
  if (tid == 0) {
    if (sm.abort) *(volatile int*)&a.cnt->abort = 1;
    if (atomicAdd(a.queue + 1, 1) == (int)gridDim.x - 1) {   // the last block out: ready for the next call
      a.queue[0] = 0;
      a.queue[1] = 0;
    }
  }
}

// ---- host --------------------------------------------------------------------
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? (EncodeTiledFn)ptr
               : (EncodeTiledFn) nullptr;
  }();
  return fn;
}

// bf16 map over [d2][d1][d0] (d0 contiguous), 128-byte swizzle, boxes of box1 x 64.
bool map3(CUtensorMap* m, const void* ptr, uint64_t d0, uint64_t d1, uint64_t d2, uint32_t box1, int rank) {
  EncodeTiledFn f = encode_fn();
  if (!f) return false;
  cuuint64_t dims[3] = {d0, d1, d2};
  cuuint64_t strides[2] = {d0 * 2, d0 * d1 * 2};
  cuuint32_t box[3] = {64, box1, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return f(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(ptr), dims, strides, box, es,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

// Buffers of partial sums: the tickets of a line that cuts tiles are no more than ticket_count gives
// for the line of every expert that can be used (make_line).
static int64_t line_units(int N, int K, int E, int nj, int kc) {
  return (N * (int64_t)K < E ? N * (int64_t)K : E) * nj * kc;
}
size_t umma_up_bytes(int N, int H, int E, int K, int F) {
  return (size_t)2 * ticket_count(line_units(N, K, E, F / 128, H / kKB), kUpTickets) * N * kPartFloats * sizeof(float);
}
size_t umma_down_bytes(int N, int H, int E, int K, int F) {
  return (size_t)2 * ticket_count(line_units(N, K, E, (H + 255) / 256, F / kKB), kDownTickets) * N * kPartFloats *
         sizeof(float);
}

moe_status experts_umma(const Args& a, const RouteCut& cut, float* part_up, float* part_down, int* tile_cnt, cudaStream_t s) {
  Params p;
  memset(&p, 0, sizeof(p));
  p.a = a;
  p.cut = cut;
  p.part_up = part_up;
  p.part_down = part_down;
  p.tile_cnt = tile_cnt;
  // both halves of the widest slot, and the up product's round16 rows of it
  const int narrow = a.N < kSplitTokens ? a.N : kSplitTokens;
  p.b_bytes[0] = 2 * (int)round_up(narrow, 8) * 128;
  p.b_bytes[1] = 2 * (int)round_up(a.N, 16) * 128;
  static_assert(2 * kSplitTokens <= 128 && kMaxTokens <= 128, "an accumulator's columns");
  size_t smem = 0;
  for (int i = 0; i < 2; ++i) {
    p.stages[i] = kSmemData / (kABytes + p.b_bytes[i]);
    if (p.stages[i] > kMaxStages) p.stages[i] = kMaxStages;
    const size_t ring = (size_t)p.stages[i] * (kABytes + p.b_bytes[i]) + 1024;
    if (smem < ring) smem = ring;
    if (a.N <= kSplitTokens) break;      // no slot is wider
  }
  if (!map3(&p.tw1, a.W1, a.F, a.H, a.E, 64, 3) || !map3(&p.tw3, a.W3, a.F, a.H, a.E, 64, 3) ||
      !map3(&p.tw2, a.W2, a.H, a.F, a.E, 64, 3) || !map3(&p.tx, a.x, a.H, a.N, 1, 1, 2) ||
      !map3(&p.tact, a.act, a.F, (uint64_t)2 * a.N * a.K, 1, 8, 2))
    return MOE_ERR_CUDA;
  static bool set[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !set[dev]) {
    if (cudaFuncSetAttribute(decode_umma_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemData + 1024) !=
            cudaSuccess ||
        cudaFuncSetAttribute(decode_umma_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemData + 1024) !=
            cudaSuccess) {
      (void)cudaGetLastError();
      return MOE_ERR_CUDA;
    }
    if (dev >= 0 && dev < 64) set[dev] = true;
  }
  cudaError_t err = cudaSuccess;
  if (a.N <= kDirectTokens)
    MOE_TRACED("decode_experts_direct", s,
               (err = launch_after(decode_umma_kernel<true>, kBlocks, kDirectThreads, smem, s, p)));
  else
    MOE_TRACED("decode_experts_umma", s, (err = launch_after(decode_umma_kernel<false>, kBlocks, kThreads, smem, s, p)));
  if (err != cudaSuccess) {
    (void)cudaGetLastError();
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // namespace decode
}  // namespace moe
