// attend_tc.cu -- paged attention for many query rows (prefill chunks, wide
// verify) on the tcgen05 tensor cores.
//
// A tile is 128 query rows (128 / group tokens times the group's heads) in
// the 128 lanes of TMEM; a block is 128 keys.  S = Q K^T lands in one of two
// 128-column buffers, a thread per row turns it into weights P in place (16
// bits, over the first half of the same columns), and O += P V takes P from
// TMEM.  Scores run two blocks ahead of the
// weights:   S0 S1 | PV0 S2 | PV1 S3 | ...
// so that the softmax of one block overlaps the products of the others.
//
// kTiles = 1 (head_dim 256, whose accumulator takes half of TMEM; or few
// rows): the two score buffers hold consecutive blocks of one tile, and two
// warpgroups take them in turn, handing on the running maximum.
// kTiles = 2 (head_dim 64, 128): the buffers hold two tiles on the same
// block, which halves the copies per product.
//
// (CTAs of a cluster do not share copies: one tile of head_dim 256 alone wants 64
// bytes a clock from L2 on every SM to keep the tensor core busy, about what the L2
// gives all SMs together, so there the copies count.)
//
// The accumulator is rescaled only when a row's maximum has grown by more
// than 2^8 since the last time (weights stay below 2^8, and the sums are
// fp32), which after the first blocks is rare; over e4m3 pages by more than 2^4.9,
// which leaves f16 weights more of their range (kLift).
//
// What bounds it: the products, 4 * 128 * 128 * head_dim flops a block and
// tile, and beside them the shared-memory traffic of their operands (Q and K
// each read per product, V once, plus the copies that bring K and V).  Over e4m3
// pages the widening comes on top of that traffic, and Q K^T waits for it.
//
// Measured with the join, 24 query and 4 key/value heads of 256: a prompt of 8192
// tokens 646 us, 1276 TFLOP/s, 66% of the burst rate of a matrix product; 2048
// tokens over 8192 keys 274 us, 1315 TFLOP/s (in e4m3 pages 511, 706); 7 tokens
// over 32771 keys in e4m3 pages 55 us.  32 heads of 128 over 8, three ragged
// chunks of 1111 over up to 20011 keys: 364 us, 1001 TFLOP/s (e4m3 499, 731).
//
// The weights are rounded to the MMA's 16 bits before P V, and the row sums add
// the unrounded ones in fp32 (attend_warp.cu).
//
// Warps: 0-3 and 4-7 softmax and output; 8 and 10 the copies of K and of V; 9
// the MMAs of P V, 12 those of Q K^T; 11 the schedule and the copies of Q.  Over
// an e4m3 cache warps 8 and 11 copy the codes of K and of V, warps 12-15 widen
// them to f16 (exact), warp 10 issues Q K^T, and the softmax warps bring their
// rows of Q, scaled by a power of two each (attend_warp.cu says why), in f16.
//
// A V value that is not finite and that only some rows of the tile see would
// reach the others as 0 * NaN: it is replaced by zero before the product and
// added to the rows that see it at the end (`dirty`).
#include <algorithm>
#include <type_traits>

#include "attend.cuh"

namespace nvfp4 {
namespace attn {
namespace {

constexpr int kM = 128;                       // rows of a tile
constexpr int kBlockShift = 7;
constexpr int kN = 1 << kBlockShift;          // keys of a block (one unit)
// Blocks that an item's beginning costs.  A prompt of 8192 tokens measured 667 us
// at 3, 646 at 4, 649 at 5 and 6; chunks of 128 over bf16 364, 364, 373, 374.
constexpr int kExtra = 4;
// Growth of log2 of a weight before rescaling, and log2 of the weight of the
// maximum that weights are taken against.  f16 ends just below 2^16 and has no
// weight below 2^-25 (attend_warp.cu says what that cost): relative error 2^-9
// down to 2^-27 of the largest, nothing lost above 2^-36.  (Slack 8 and lift 7
// rescale less often, chunks of 128 497 us against 503, but 2^-27 would have an
// error of 2^-5.)
template <bool kE4m3>
constexpr float kSlack = kE4m3 ? 4.9375f : 8.f;
template <bool kE4m3>
constexpr float kLift = kE4m3 ? 11.f : 0.f;
// Registers of a thread in the softmax warps and in the others: in all what 512
// threads of 128 registers are launched with.
constexpr int kSoftmaxRegs = 192, kHelperRegs = 64;
constexpr int kRawBytes = 8 * 1024;           // of a unit of e4m3 codes
constexpr int kItems = 4;                     // item descriptors in flight
constexpr int kDirty = 8;                     // items whose `dirty` note is held: more than the ring's

template <int kDim, bool kE4m3, int kTiles>
struct Cfg {
  static constexpr int kThreads = 512;
  // A slot holds up to 32 KB: 128 of head_dim of all keys of a K block, or all
  // of head_dim of some keys of a V block, in chunks of 64 columns.
  static constexpr int kSlotBytes = std::min(kDim * kN * 2, 32 * 1024);
  static constexpr int kPieces = kDim * kN * 2 / kSlotBytes;   // slots of one K (or V) block
  static constexpr int kKChunks = kDim / 64 / kPieces;         // of a K slot
  static constexpr int kKChunk = kN * 128;                     // bytes of one of them
  static constexpr int kVChunks = kDim / 64;                   // of a V slot
  static constexpr int kVKeys = kN / kPieces;
  static constexpr int kVChunk = kVKeys * 128;
  static constexpr int kQTile = kM * kDim * 2;
  static constexpr int kQBytes = kTiles * kQTile;
  static constexpr int kMaxSlots = 8;
  static constexpr int kBars = 2 * kMaxSlots + 32 + 2 * kItems;
  static constexpr int kBarOff = 0;
  static constexpr int kItemOff = (kBarOff + kBars * 8 + 16 + kDirty * 4 + 15) / 16 * 16;  // descriptors
  static constexpr int kMaxOff = kItemOff + kItems * 32;                                   // running maxima
  static constexpr int kSumOff = kMaxOff + (kTiles == 1 ? kM * 4 : 0);        // row sums
  static constexpr int kFixed = kSumOff + (kTiles == 1 ? kM * 4 : 0);
  // e4m3 codes on their way: two units of K, two of V
  static constexpr int kRaw = kE4m3 ? 4 * kRawBytes : 0;
  static constexpr int kBudget = 227 * 1024 - 1024 - kFixed - kQBytes - kRaw;
  static constexpr int kSlots = std::min(kMaxSlots, kBudget / kSlotBytes);
  static constexpr int kSmem = kQBytes + kRaw + kSlots * kSlotBytes + kFixed + 1024;
  // K and V have rings of their own, since different warps fill them.  K slots
  // come free, and are filled again, while V is in use, and V's while K is.
  static constexpr int kKSlots = kSlots / 2, kVSlots = kSlots - kKSlots;
  static_assert(kKSlots >= kPieces, "K and V of one block have to fit");
  static_assert(kSlots * kSlotBytes >= static_cast<int>(sizeof(RangeSmem)), "scratch of the start");
  // TMEM columns: the accumulators, then the two score buffers
  static constexpr uint32_t kO = 0;
  static constexpr uint32_t kS = kTiles * kDim;
  static_assert(kS + 2 * kN <= 512, "TMEM");
};

template <bool kE4m3>
__device__ __forceinline__ uint32_t idesc(uint32_t n, bool b_mn_major) {
  return (kE4m3 ? umma_idesc_f16(kM, n) : umma_idesc_bf16(kM, n)) | (b_mn_major ? 1u << 16 : 0u);
}

__device__ __forceinline__ void tmem_st_16cols(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// One 32-byte store (a whole sector): the rows of a warp's lanes lie far apart,
// and two 16-byte halves would be two transactions.
__device__ __forceinline__ void st_global_32(void* at, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Four e4m3 codes as two f16x2: exact.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t v, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(v));
}

// Whether any of a word's two 16-bit values is not finite.
template <bool kE4m3>
__device__ __forceinline__ bool non_finite(uint32_t w) {
  constexpr uint32_t e = kE4m3 ? 0x7C00u : 0x7F80u;
  return (w & e) == e || (w & (e << 16)) == (e << 16);
}
template <bool kE4m3>
__device__ __forceinline__ uint32_t finite_mask(uint32_t w) {
  constexpr uint32_t e = kE4m3 ? 0x7C00u : 0x7F80u;
  return ((w & e) == e ? 0u : 0xFFFFu) | ((w & (e << 16)) == (e << 16) ? 0u : 0xFFFF0000u);
}

// A position in a ring of slots, of which the first is `kFirst`, and the parity
// of its turn.
template <int kFirst, int kSlots>
struct Ring {
  int slot = kFirst;
  uint32_t par = 0;
  __device__ void next() {
    if (++slot == kFirst + kSlots) slot = kFirst, par ^= 1u;
  }
};

struct TcParams {
  Attend a;
  Plan plan;
  Parts parts;
  int tile_tokens;          // tokens of one 128-row tile
  int box_shift;            // log2 of the slots of one page copy
};

// One item of the CTA's range, as the scheduling lane publishes it to the other
// warps (the code that finds the next item exists once: inlined in every role
// it made the kernel larger than the instruction cache, and every role's
// steps several times slower).
struct alignas(16) Item {
  int s, h, q0, q_len, kv_len;
  int tok0;                   // first token, of the sequence's new ones
  int key0;                   // first key
  int blocks;                 // 0: the end of the range; kBegins, kEnds in its top bits
  __device__ int count() const { return blocks & 0x0FFFFFFF; }
  // keys that every token sees, that the last token sees
  __device__ int least() const { return max(0, kv_len - q_len + tok0 + 1); }
  __device__ int seen(const Plan& p) const {
    return max(0, kv_len - q_len + min(q_len, tok0 + p.tile_tokens));
  }
};
constexpr int kBegins = 1 << 30, kEnds = 1 << 29;

struct Items {
  Item* ring;
  uint64_t* full;
  uint64_t* empty;
  volatile int* abort_flag;
  // Item i, or false at the end (or when waiting for it was given up).
  __device__ bool get(int i, Item& it) const {
    const bool ok = wait(&full[i % kItems], i / kItems & 1, abort_flag);
    const int4* src = reinterpret_cast<const int4*>(&ring[i % kItems]);
    reinterpret_cast<int4*>(&it)[0] = src[0];
    reinterpret_cast<int4*>(&it)[1] = src[1];
    if (!ok) it.blocks = 0;
    return it.blocks != 0;
  }
  // One role is done with item i.
  __device__ void release(int i) const { mbar_arrive(&empty[i % kItems]); }
};

// A role's place in the sequence of blocks.
struct Place {
  Item it;
  int item = 0, b = 0;
  bool live;
  __device__ void start(const Items& items) { live = items.get(0, it); }
  __device__ bool first() const { return b == 0; }
  __device__ bool last() const { return b + 1 == it.count(); }
  // To the next block; true where it is another item's.
  __device__ bool next(const Items& items) {
    if (++b < it.count()) return false;
    b = 0;
    live = items.get(++item, it);
    return true;
  }
};

// How the widening warps of K or V cut a block: units of 8 passes by 64 threads.
template <class C, int kDim, bool kV>
struct Units {
  static constexpr int kSlotRows = kV ? C::kVKeys : kN;
  static constexpr int kPerRow = kV ? kDim / 16 : C::kKChunks * 4;    // threads of a row
  static constexpr int kRowsAtOnce = 64 / kPerRow;
  static constexpr int kPasses = 8;
  static constexpr int kRows = kPasses * kRowsAtOnce;
  static constexpr int kRowShift = kRows == 128 ? 7 : kRows == 64 ? 6 : 5;
  static constexpr int kHalves = kSlotRows / kRows;                   // units of a slot
  static constexpr int kCount = C::kPieces * kHalves;                 // of a block
  static constexpr int kKeyUnits = kN / kRows;                        // of different keys
  static constexpr int kWidth = kDim < 128 ? 64 : 128;                // bytes of a row's copy
  static constexpr int kChunks = kV && kDim == 256 ? 2 : 1;           // copies of a row
  static_assert(kRows * kPerRow * 16 == kRawBytes && (1 << kRowShift) == kRows, "a unit's bytes");
};

template <class C>
using KRing = Ring<0, C::kKSlots>;
template <class C>
using VRing = Ring<C::kKSlots, C::kVSlots>;

template <int kDim, bool kE4m3, int kTiles>
__global__ void __launch_bounds__(Cfg<kDim, kE4m3, kTiles>::kThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                     const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const TcParams p) {
  using C = Cfg<kDim, kE4m3, kTiles>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* q_sm = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* raw = q_sm + C::kQBytes;                // [K, V][2]
  uint8_t* ring = raw + C::kRaw;
  uint8_t* fixed = ring + C::kSlots * C::kSlotBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(fixed + C::kBarOff);
  uint64_t* empty = full + C::kMaxSlots;
  uint64_t* s_full = empty + C::kMaxSlots;        // [2] scores in buffer x
  uint64_t* p_full = s_full + 2;                  // [2][2] weights in buffer x, by halves of the keys
  uint64_t* pv_done = p_full + 4;                 // [2] product with buffer x's weights
  uint64_t* o_free = pv_done + 2;                 // [2] accumulator read out
  uint64_t* m_ready = o_free + 2;                 // [2][4] running maximum handed on, per warp
  uint64_t* q_full = m_ready + 8;
  uint64_t* q_empty = q_full + 1;
  uint64_t* mma_done = q_empty + 1;               // every product issued has completed
  uint64_t* pair = mma_done + 1;                  // both softmax groups (kTiles == 1)
  uint64_t* raw_full = pair + 1;                  // [K, V][2] (e4m3)
  uint64_t* raw_free = raw_full + 4;
  uint64_t* v_known = raw_free + 4;                  // [2] v_slot[x] is that of buffer x's block
  const Items items{reinterpret_cast<Item*>(fixed + C::kItemOff), v_known + 2, v_known + 2 + kItems,
                    reinterpret_cast<volatile int*>(full + C::kBars)};
  volatile int* abort_flag = reinterpret_cast<volatile int*>(full + C::kBars);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + C::kBars) + 1;
  volatile int* v_slot = reinterpret_cast<volatile int*>(full + C::kBars) + 2; // [2] slot, parity << 8
  volatile int* dirty = v_slot + 2;               // [kDirty] item ordinal + 1
  float* run_max = reinterpret_cast<float*>(fixed + C::kMaxOff);
  float* row_sum = reinterpret_cast<float*>(fixed + C::kSumOff);
  const Attend& a = p.a;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kSlots; ++i) {
      mbar_init(&full[i], kE4m3 ? 2 : 1);
      mbar_init(&empty[i], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[2 * x], 4);
      mbar_init(&p_full[2 * x + 1], 4);
      mbar_init(&pv_done[x], 1);
      mbar_init(&v_known[x], 1);
      mbar_init(&o_free[x], kTiles == 1 ? 8 : 4);
      for (int i = 0; i < 4; ++i) mbar_init(&m_ready[x * 4 + i], 1);
    }
    mbar_init(q_full, kE4m3 ? 8 : 1);
    for (int i = 0; i < 4; ++i) mbar_init(&raw_full[i], 1), mbar_init(&raw_free[i], 2);
    mbar_init(q_empty, 1);
    mbar_init(mma_done, 2);
    mbar_init(pair, 8);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(&items.full[i], 1);
      // softmax, MMA, copying and widening warps
      mbar_init(&items.empty[i], 8 + 2 + (kE4m3 ? 2 + 4 : 2));
    }
    *abort_flag = 0;
    for (int i = 0; i < kDirty; ++i) dirty[i] = 0;
    fence_mbar_init();
    if (!kE4m3) prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();
  // the range, in scratch that the ring's first copies will overwrite
  const Range range =
      find_range(a.seqs, a.cache.heads, p.plan, blockIdx.x, gridDim.x,
                 reinterpret_cast<RangeSmem*>(ring), a.err);
  fence_proxy_async_smem();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_slot;

  // The scheduling lane: item i, or the end, to all other warps; false at the end.
  auto publish = [&](const Walk& w, int i) {
    if (i >= kItems && !wait(&items.empty[i % kItems], (i / kItems & 1) ^ 1, abort_flag))
      return false;
    Item it{};
    if (w.more())
      it = Item{w.r.s, w.r.h, w.seq.q0, w.seq.q_len, w.seq.kv_len, w.r.tile * p.plan.tile_tokens,
                w.unit0 * kN, w.count | (w.begins() ? kBegins : 0) | (w.ends() ? kEnds : 0)};
    items.ring[i % kItems] = it;
    mbar_arrive(&items.full[i % kItems]);
    return w.more();
  };

  // Of a V slot whose first key is key0, rows row0 to row0 + rows - 1, as far as
  // not all rows of the tile see them: rows that none sees become zero (0 times
  // what a page happens to hold past the length need not be 0), and values that
  // are not finite do; whether there were any.  By one warp.
  auto check_rows = [&](const Item& it, int key0, int slot, int row0, int rows) {
    constexpr int kPer = C::kVChunks * 8;                   // 16-byte pieces of a row
    const int least = it.least(), seen = it.seen(p.plan);
    const int from = max(row0, least - key0);
    bool bad = false;
#pragma unroll 1
    for (int j = from * kPer + lane; j < (row0 + rows) * kPer; j += 32) {
      uint4* at = reinterpret_cast<uint4*>(ring + slot * C::kSlotBytes +
                                           (j % kPer >> 3) * C::kVChunk + j / kPer * 128 +
                                           (j & 7) * 16);
      if (key0 + j / kPer >= seen) {
        *at = make_uint4(0, 0, 0, 0);
        continue;
      }
      uint4 v = *at;
      if (!(non_finite<kE4m3>(v.x) || non_finite<kE4m3>(v.y) || non_finite<kE4m3>(v.z) ||
            non_finite<kE4m3>(v.w)))
        continue;
      bad = true;
      v.x &= finite_mask<kE4m3>(v.x), v.y &= finite_mask<kE4m3>(v.y);
      v.z &= finite_mask<kE4m3>(v.z), v.w &= finite_mask<kE4m3>(v.w);
      *at = v;
    }
    return bad;
  };
  // All of block b, a quarter by each warp of the group that gives its weights.
  auto check_v = [&](const Item& it, int b, int at, int quad) {
    constexpr int kRows = C::kVKeys / 4;
    VRing<C> r;
    r.slot = at & 255, r.par = at >> 8;
    bool bad = false;
#pragma unroll 1
    for (int h = 0; h < C::kPieces; ++h, r.next()) {
      wait(&full[r.slot], r.par, abort_flag);
      __syncwarp();
      bad |= check_rows(it, it.key0 + b * kN + h * C::kVKeys, r.slot, quad * kRows, kRows);
    }
    fence_proxy_async_smem();
    return bad;
  };

  // One warp for the copies of K, one for those of V.  Each lane keeps the
  // operands of one copy of a block (piece, rows, chunks), its page read one
  // block ahead, so that a slot costs a wait and an issue: one warp's dependent
  // instructions are what the copies would otherwise wait for.
  auto copy_pages = [&](auto values) {
    constexpr bool kV = decltype(values)::value;
    constexpr int kRows = kV ? C::kVKeys : kN;              // of a slot
    constexpr int kChunks = kV ? C::kVChunks : C::kKChunks; // of a slot
    constexpr int kRowShift = kRows == 128 ? 7 : 6;
    const CUtensorMap* map = kV ? &tm_v : &tm_k;
    const int shift = min(p.box_shift, kRowShift);          // log2 of the rows of a copy
    const int boxes = kRows >> shift;
    const int at_once = kV && boxes == 1 ? kChunks : 1;     // chunks of a copy
    // lane: copy (box, chunk) of each slot; of V also the slot, whose keys differ
    const int per_slot = boxes * (kChunks / at_once);
    const int piece = kV ? lane / per_slot : 0;
    const int box = lane % per_slot / (kChunks / at_once);
    const int chunk = lane % (kChunks / at_once) * at_once;
    const bool has_copy = lane < (kV ? C::kPieces : 1) * per_slot;
    const int row = (kV ? piece * kRows : 0) + (box << shift);
    const uint32_t dst = chunk * (kRows * 128) + (box << (shift + 7));
    const uint32_t bytes = at_once << (shift + 7);
    Place at;
    at.start(items);
    __syncwarp();
    std::conditional_t<kV, VRing<C>, KRing<C>> r;
    constexpr int kTurns = kV ? C::kVSlots : C::kKSlots;
    int turns = 0;                                          // slots filled, up to kTurns
    bool ok = true;
    int key = 0, entry = 0;
    auto look_up = [&]() {
      key = at.it.key0 + at.b * kN + row;
      if (at.live && has_copy && key < at.it.kv_len)
        entry = a.seqs.table[int64_t(at.it.s) * a.seqs.width + key / a.cache.page_size];
      else
        key = -1;
    };
    look_up();
    while (ok && at.live) {
      int page = -1, in_page = 0;
      if (key >= 0) {
        page = static_cast<int>(checked_page(entry, a.cache.pages, a.err));
        in_page = key % a.cache.page_size;
      }
      const int head = at.it.h, was = at.item;
      const bool moved = at.next(items);
      __syncwarp();
      if (moved && lane == 0) items.release(was);
      look_up();
      for (int h = 0; h < C::kPieces; ++h, r.next()) {
        const bool mine = page >= 0 && (!kV || piece == h);
        const int n = __popc(__ballot_sync(0xffffffffu, mine));
        if (turns == kTurns)
          ok = __all_sync(0xffffffffu, wait(&empty[r.slot], r.par ^ 1, abort_flag));
        else
          ++turns;
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&full[r.slot], n * bytes);
        __syncwarp();
        if (mine)
          tma_load_page(ring + r.slot * C::kSlotBytes + dst, map, &full[r.slot],
                        (kV ? 0 : h * kChunks) + chunk, in_page, head, page);
      }
    }
    // every copy has landed before the block may end
    const int first = kV ? C::kKSlots : 0;
    for (int s = first; s < first + turns; ++s) {
      volatile int no_abort = 0;
      if (!wait(&full[s], s < r.slot ? r.par : r.par ^ 1, &no_abort))
        atomicOr(a.err, NVFP4_ATTENTION_TIMEOUT);
    }
    __syncwarp();
  };

  // e4m3 codes of K or of V, unit by unit (a unit: 8 KB, what 64 threads widen in
  // 8 passes), copied by one warp into two buffers.  Each lane keeps the operands
  // of one copy of a block (unit, box, chunk), its page read one block ahead.
  // `moved(item)`: called when the item before `item` is done with.
  auto copy_raw = [&](auto values, auto moved) {
    constexpr bool kV = decltype(values)::value;
    using U = Units<C, kDim, kV>;
    const CUtensorMap* map = kV ? &tm_v : &tm_k;
    const int shift = min(p.box_shift, U::kRowShift);
    // a row's chunks: in one copy, where that has all rows of the unit
    const int chunks = (1 << shift) == U::kRows ? 1 : U::kChunks;
    const int per_unit = (U::kRows >> shift) * chunks;
    const int unit = lane / per_unit, box = lane % per_unit / chunks, chunk = lane % chunks;
    const bool has_copy = unit < U::kKeyUnits;
    const int row = unit * U::kRows + (box << shift);
    const int bytes = (U::kWidth << shift) * (U::kChunks / chunks);
    const uint32_t dst = chunk * U::kRows * U::kWidth + (box << shift) * U::kWidth;
    uint64_t* bar = raw_full + (kV ? 2 : 0);
    uint64_t* free = raw_free + (kV ? 2 : 0);
    Place at;
    at.start(items);
    __syncwarp();
    bool ok = true;
    int count = 0, key = -1, entry = 0;
    auto look_up = [&]() {
      key = at.it.key0 + at.b * kN + row;
      if (at.live && has_copy && key < at.it.kv_len)
        entry = a.seqs.table[int64_t(at.it.s) * a.seqs.width + key / a.cache.page_size];
      else
        key = -1;
    };
    look_up();
    while (ok && at.live) {
      int page = -1, in_page = 0;
      if (key >= 0) {
        page = static_cast<int>(checked_page(entry, a.cache.pages, a.err));
        in_page = key % a.cache.page_size;
      }
      const int head = at.it.h, was = at.item;
      const bool next_item = at.next(items);
      __syncwarp();
      look_up();
#pragma unroll 1
      for (int u = 0; u < U::kCount; ++u, ++count) {
        const int b = count & 1;
        const bool mine = page >= 0 && unit == u % U::kKeyUnits;
        const int n = __popc(__ballot_sync(0xffffffffu, mine));
        if (count >= 2)
          ok = __all_sync(0xffffffffu, wait(&free[b], (count >> 1 & 1) ^ 1, abort_flag));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(&bar[b], n * bytes);
        __syncwarp();
        if (mine)
          tma_load_page(raw + ((kV ? 2 : 0) + b) * kRawBytes + dst, map, &bar[b],
                        u / U::kKeyUnits + chunk, in_page, head, page);
      }
      if (ok && next_item) {
        if (lane == 0) items.release(was);
        moved(was + 1);
      }
    }
    // every copy has landed before the block may end
    for (int i = max(0, count - 2); i < count; ++i) {
      volatile int no_abort = 0;
      if (!wait(&bar[i & 1], i >> 1 & 1, &no_abort)) atomicOr(a.err, NVFP4_ATTENTION_TIMEOUT);
    }
    __syncwarp();
  };

  // Two warps widen K, two V: a thread's 16 codes become 32 bytes of the slot.
  // (Codes loaded from the pages to registers held up every arrival and fence,
  // which wait for the loads before them.)
  auto widen_pages = [&](auto values) {
    constexpr bool kV = decltype(values)::value;
    using U = Units<C, kDim, kV>;
    constexpr int kChunkBytes = kV ? C::kVChunk : C::kKChunk;
    constexpr int kRowsAtOnce = U::kRowsAtOnce;
    // Four lanes take 64 codes of a row and the next four those of another row,
    // whose number differs in bits 0 and 2: so that of eight lanes neither the
    // loads nor the stores meet in a bank.  (All eight in one row: their stores
    // meet, pass time 850 to 1080 clocks.)
    const int tid = threadIdx.x & 63, odd = U::kPerRow >= 8 ? tid >> 2 & 1 : 0;
    const int my_row = U::kPerRow == 16  ? (tid >> 5) * 2 + odd
                       : U::kPerRow == 8 ? (tid >> 4 & 1) * 4 + (tid >> 5) * 2 + odd
                                         : tid / U::kPerRow;
    const int my_col = U::kPerRow == 16  ? ((tid >> 3 & 3) * 4 + (tid & 3)) * 16
                       : U::kPerRow == 8 ? ((tid >> 3 & 1) * 4 + (tid & 3)) * 16
                                         : tid % U::kPerRow * 16;
    // consecutive rows of a slot that one of the two warps writes, and their distance
    constexpr int kRun = U::kPerRow >= 8 ? 2 : kRowsAtOnce / 2;
    // where a pass's 16 bytes come from in the unit, and its 32 bytes go in the
    // slot: both swizzles repeat every 8 rows
    const int c16 = (my_col & 63) >> 3;
    uint32_t get[2], put[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int rr = (i * kRowsAtOnce + my_row) ^ (odd << 2);
      get[i] = U::kWidth == 128
                   ? (my_col >> 7) * U::kRows * 128 + rr * 128 + (((my_col & 127) >> 4 ^ (rr & 7)) << 4)
                   : rr * 64 + ((my_col >> 4 ^ (rr >> 1 & 3)) << 4);
#pragma unroll
      for (int k = 0; k < 2; ++k)
        put[i][k] = (my_col >> 6) * kChunkBytes + rr * 128 + (((c16 + k) ^ (rr & 7)) << 4);
    }
    Place at;
    at.start(items);
    __syncwarp();
    std::conditional_t<kV, VRing<C>, KRing<C>> r;
    int turns = 0;                                               // slots filled, up to the ring's
    int count = 0;                                               // units widened
    while (at.live) {
      const int key0 = at.it.key0 + at.b * kN;
#pragma unroll 1
      for (int u = 0; u < U::kCount; ++u, ++count) {
        if (u % U::kHalves == 0) {
          if (turns == (kV ? C::kVSlots : C::kKSlots)) {
            wait(&empty[r.slot], r.par ^ 1, abort_flag);
            __syncwarp();
          } else {
            ++turns;
          }
        }
        const int b = (kV ? 2 : 0) + (count & 1);
        wait(&raw_full[b], count >> 1 & 1, abort_flag);
        __syncwarp();
        const uint8_t* unit = raw + b * kRawBytes;
        uint8_t* slot = ring + r.slot * C::kSlotBytes + (u % U::kHalves) * U::kRows * 128;
#pragma unroll
        for (int i = 0; i < U::kPasses; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(unit + (i >> 1) * (2 * kRowsAtOnce * U::kWidth) + get[i & 1]);
          uint32_t f[8];
          e4m3x4_to_f16x4(v.x, f[0], f[1]);
          e4m3x4_to_f16x4(v.y, f[2], f[3]);
          e4m3x4_to_f16x4(v.z, f[4], f[5]);
          e4m3x4_to_f16x4(v.w, f[6], f[7]);
          uint8_t* at_row = slot + (i >> 1) * (2 * kRowsAtOnce * 128);
          *reinterpret_cast<uint4*>(at_row + put[i & 1][0]) = make_uint4(f[0], f[1], f[2], f[3]);
          *reinterpret_cast<uint4*>(at_row + put[i & 1][1]) = make_uint4(f[4], f[5], f[6], f[7]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&raw_free[b]);
        if (u % U::kHalves == U::kHalves - 1) {
          // the passes' rows of a V slot lie with both warps: each looks over the
          // rows that it wrote
          const int first = key0 + u / U::kHalves * (U::kRows * U::kHalves);
          if (kV && first + U::kRows * U::kHalves > at.it.least()) {
            bool bad = false;
#pragma unroll 1
            for (int q = 0; q < U::kRows * U::kHalves; q += 2 * kRun)
              bad |= check_rows(at.it, first, r.slot, q + (warp & 1) * kRun, kRun);
            if (bad) dirty[at.item % kDirty] = at.item + 1;
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full[r.slot]);
          r.next();
        }
      }
      const int was = at.item;
      const bool moved = at.next(items);
      __syncwarp();
      if (moved && lane == 0) items.release(was);
    }
  };

  // A softmax thread's query row, scaled by a power of two, in f16; what the
  // row's scores have to be multiplied by.  With one tile the thread of either
  // group stores half of the columns.  (A lane per row keeps this to two short
  // loops: unrolled over rows it was 28 KB of code that runs once, and fetching
  // it took 10 us.)
  auto scale_row = [&](const Item& it, int x, int row, bool valid) {
    // a row that holds no token is left as it is: its weights are 0
    if (!valid) return 1.f;
    const int tok = row / a.group, gi = row - tok * a.group, tile = kTiles == 2 ? x : 0;
    const int ti = it.tok0 + tile * p.tile_tokens + tok;
    const uint4* src = reinterpret_cast<const uint4*>(
        a.q.data + int64_t(it.q0 + ti) * a.q.ts + int64_t(it.h * a.group + gi) * a.q.hs);
    uint32_t top2 = 0;                                  // magnitudes order as integers
#pragma unroll 8
    for (int k = 0; k < kDim / 8; ++k) {
      const uint4 v = src[k];
      top2 = max_u16x2(max_u16x2(top2, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
      top2 = max_u16x2(max_u16x2(top2, v.z & 0x7FFF7FFFu), v.w & 0x7FFF7FFFu);
    }
    const uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
    const int e = top == 0 || top >= 0x7F80u ? 0 : min(141 - static_cast<int>(top >> 7), 100);
    const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    constexpr int kPieces = kDim / 8 / (kTiles == 1 ? 2 : 1);
    const int k0 = kTiles == 1 ? x * kPieces : 0;
    uint8_t* dst = q_sm + tile * C::kQTile + row * 128;
#pragma unroll 2
    for (int k = k0; k < k0 + kPieces; ++k) {
      const uint4 v = src[k];
      const uint32_t in[4] = {v.x, v.y, v.z, v.w};
      uint32_t f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = f32x2_to_f16x2(bf16_lo(in[i]) * up, bf16_hi(in[i]) * up);
      // elements 8 k on: 64-column chunk k / 8, 16-byte piece k % 8 of the row
      *reinterpret_cast<uint4*>(dst + (k >> 3) * kM * 128 + (((k & 7) ^ (row & 7)) << 4)) =
          make_uint4(f[0], f[1], f[2], f[3]);
    }
    return __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  };

  const bool lead = lane == 0;
  constexpr int kScoreWarp = kE4m3 ? 10 : 12;
  // Nothing may be in flight when TMEM is released.
  auto drain = [&]() {
    if (lead) {
      umma_commit(mma_done);
      volatile int no_abort = 0;
      if (!wait(mma_done, 0, &no_abort)) atomicOr(a.err, NVFP4_ATTENTION_TIMEOUT);
    }
    __syncwarp();
  };
  // MMA: S = Q K^T.  A warp of its own: an issue waits for the pipe, so that what
  // one warp spends between its products the other's have to fill.
  auto score_mma = [&]() {
    const uint32_t id_s = idesc<kE4m3>(kN, false);
    const uint32_t q_lo = desc_lo(smem_addr(q_sm), 0);
    const uint32_t k_lo = desc_lo(smem_addr(ring), 0);
    Place qk;
    int x = 0;                                  // the score buffer (and tile)
    qk.start(items);
    KRing<C> next, at;                          // of the next block; of the one in use
    bool ok = true;
    auto ready = [&](uint64_t* bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, wait(bar, parity, abort_flag));
    };
    for (int i = 0; ok && qk.live; ++i, x ^= 1) {
      const uint32_t t_s = tmem + C::kS + x * kN;
      if (kTiles == 1 || x == 0) {
        if (qk.first()) ready(q_full, qk.item & 1);
        at = next;
#pragma unroll
        for (int h = 0; h < C::kPieces; ++h) next.next();
      }
      // the weights that the buffer held have been used
      if (i >= 2) ready(&pv_done[x], (i >> 1 & 1) ^ 1);
      KRing<C> r = at;
      const uint32_t q = q_lo + (kTiles == 2 ? x * (C::kQTile >> 4) : 0);
      const bool last = qk.last() && (kTiles == 1 || x == 1);
#pragma unroll 1
      for (int h = 0; h < C::kPieces; ++h, r.next()) {
        if (kTiles == 1 || x == 0) ready(&full[r.slot], r.par);
        if (!ok) break;
        tc_fence_after_sync();
        if (lead) {
          const uint32_t k = k_lo + r.slot * (C::kSlotBytes >> 4);
          const uint32_t qh = q + h * ((C::kKChunks * C::kKChunk) >> 4);
          const uint32_t acc = h != 0;
#pragma unroll
          for (int kk = 0; kk < C::kKChunks * 4; ++kk) {
            const uint32_t off = ((kk >> 2) * C::kKChunk + (kk & 3) * 32) >> 4;
            umma_ss(t_s, qh + off, k + off, id_s, kk == 0 ? acc : 1u);
          }
          if (kTiles == 1 || x == 1) umma_commit(&empty[r.slot]);
          if (h == C::kPieces - 1) {
            umma_commit(&s_full[x]);
            if (last) umma_commit(q_empty);
          }
        }
        __syncwarp();
      }
      if (ok && (kTiles == 1 || x == 1)) {
        const int was = qk.item;
        if (qk.next(items) && lead) items.release(was);
        __syncwarp();
      }
    }
    drain();
  };

  if (warp < 8) {
    // ------------------------------------------------------ softmax, output
    regs_inc<kSoftmaxRegs>();
    const int x = warp >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;                 // of the tile
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t t_s = lane_base + C::kS + x * kN;
    const uint32_t t_o = lane_base + C::kO + (kTiles == 2 ? x * kDim : 0);
    const int tok = row / a.group, gi = row - tok * a.group;
    int flags = 0;
    int4 note = make_int4(0, 0, 0, 0);
    int step = 0;                                     // of both buffers (kTiles == 1)
    int uses = 0;                                     // of buffer x
    uint32_t pair_par = 0;
    auto meet = [&]() {                               // both groups
      __syncwarp();
      if (lane == 0) mbar_arrive(pair);
      wait(pair, pair_par, abort_flag);
      __syncwarp();
      pair_par ^= 1u;
    };
    Item it;
    for (int item = 0; items.get(item, it); ++item) {
      __syncwarp();
      const int ti = it.tok0 + (kTiles == 2 ? x : 0) * p.tile_tokens + tok;
      const bool valid = tok < p.tile_tokens && ti < it.q_len;
      const int lim = valid ? max(0, it.kv_len - it.q_len + ti + 1) : 0;
      const int count = it.count();
      float c = a.scale * 1.44269504088896f;
      if constexpr (kE4m3) {
        if (a.cache.k_scale) c *= a.cache.k_scale[it.h];
        if (item > 0) wait(q_empty, (item - 1) & 1, abort_flag);
        __syncwarp();
        c *= scale_row(it, x, row, valid);
        __syncwarp();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(q_full);
      }
      float m = -INFINITY, l = 0.f;                   // of the blocks that this thread saw
      for (int b = 0; b < count; ++b, ++step) {
        if (kTiles == 1 && (step & 1) != x) continue;
        float prev = m;                               // the maximum before this block
        if (kTiles == 1 && b > 0) {
          wait(&m_ready[(x ^ 1) * 4 + quad], ((step - 1) >> 1) & 1, abort_flag);
          __syncwarp();
          prev = run_max[row];
        }
        wait(&s_full[x], uses & 1, abort_flag);
        __syncwarp();
        tc_fence_after_sync();
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld_32cols(t_s + i * 32, s[i]);
        tmem_ld_wait();
        const int seen = lim - it.key0 - b * kN;      // of this block, by this row
        if (__any_sync(0xffffffffu, seen < kN)) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (i * 32 + j >= seen) s[i][j] = 0xFF800000u;
        }
        float t4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          t4[i] = fmaxf(__uint_as_float(s[i][0]), __uint_as_float(s[i][1]));
#pragma unroll
          for (int j = 2; j < 32; j += 2)
            t4[i] = fmaxf(t4[i], fmaxf(__uint_as_float(s[i][j]), __uint_as_float(s[i][j + 1])));
        }
        const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * c;
        // ---- the maximum the weights are taken against
        float now = top;
        if (b > 0) {
          now = fmaxf(prev, top);
          if (__any_sync(0xffffffffu, now - prev > kSlack<kE4m3>)) {
            // the accumulator, complete up to the block before
            if (kTiles == 1)
              wait(&pv_done[x ^ 1], ((step - 1) >> 1) & 1, abort_flag);
            else
              wait(&pv_done[x], (uses - 1) & 1, abort_flag);
            __syncwarp();
            tc_fence_after_sync();
            const float alpha = prev == -INFINITY ? 0.f : ex2(prev - now);
#pragma unroll 1
            for (int i = 0; i < kDim; i += 32) {
              uint32_t o[32];
              tmem_ld_32cols(t_o + i, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
              tmem_st_32cols(t_o + i, o);
            }
            tmem_st_wait();
          } else {
            now = prev;
          }
        }
        if (kTiles == 1) {
          run_max[row] = now;
          __syncwarp();
          if (lane == 0) mbar_arrive(&m_ready[x * 4 + quad]);
        }
        const float base = now == -INFINITY ? 0.f : now;
        if (m != now) l *= m == -INFINITY ? 0.f : ex2(m - base);
        m = now;
        if (!kE4m3 && (kTiles == 1 || x == 0) && it.key0 + (b + 1) * kN > it.least()) {
          wait(&v_known[x], uses & 1, abort_flag);
          __syncwarp();
          if (check_v(it, b, v_slot[x], quad)) dirty[item % kDirty] = item + 1;
        }
        // ---- the weights, handed over by halves
        const float2 c2 = make_float2(c, c), b2 = make_float2(kLift<kE4m3> - base, kLift<kE4m3> - base);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w16[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float2 e = fma2(make_float2(__uint_as_float(s[i][2 * j]), __uint_as_float(s[i][2 * j + 1])),
                            c2, b2);
            e.x = ex2(e.x), e.y = ex2(e.y);
            sum[j & 1] = add2(sum[j & 1], e);
            w16[j] = kE4m3 ? f32x2_to_f16x2(e.x, e.y) : f32x2_to_bf16x2(e.x, e.y);
          }
          tmem_st_16cols(t_s + i * 16, w16);
          if (i & 1) {
            tmem_st_wait();
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[2 * x + (i >> 1)]);
          }
        }
        sum[0] = add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;
        ++uses;
      }
      // ---- the row's sum, and the result
      const bool whole = (it.blocks & kBegins) && (it.blocks & kEnds);
      const int part = it.blocks & kBegins ? 1 : 0;
      if (!whole) {
        flags |= part ? kPart1 : kPart0 | (it.blocks & kEnds ? kPart0Ends : 0);
        if (part) note = make_int4(0, it.s, it.h, it.tok0 / p.plan.tile_tokens);
      }
      if (kTiles == 1) {
        // The last block's maximum, and the last product, whose weights both groups
        // gave.  The group that did not give the last block's waits for its maximum
        // first: only then is the product two blocks before known to have completed,
        // and the parity of the last one's barrier that of no earlier phase.
        if (((step - 1) & 1) != x) {
          wait(&m_ready[(x ^ 1) * 4 + quad], ((step - 1) >> 1) & 1, abort_flag);
          __syncwarp();
        }
        wait(&pv_done[(step - 1) & 1], ((step - 1) >> 1) & 1, abort_flag);
        __syncwarp();
        const float now = run_max[row];               // of the last block
        if (m != -INFINITY) l *= ex2(m - now);
        meet();                                       // both groups have read it
        float* mine = x ? row_sum : run_max;
        const float* other = x ? run_max : row_sum;
        mine[row] = l;
        meet();
        l = x ? other[row] + l : l + other[row];
        m = now;
      } else {
        wait(&pv_done[x], (uses - 1) & 1, abort_flag);
        __syncwarp();
      }
      tc_fence_after_sync();
      const float vs = kE4m3 && a.cache.v_scale ? a.cache.v_scale[it.h] : 1.f;
      const float inv = l == 0.f ? 0.f : vs / l;
      const int64_t token = it.q0 + ti;
      const int head = it.h * a.group + gi;
      const int64_t at_part = p.parts.row(blockIdx.x, part, (kTiles == 2 ? x * kM : 0) + row);
      if (valid && (kTiles == 2 || x == 0)) {
        const float lse2 = l == 0.f ? -INFINITY : m + (log2f(l) - kLift<kE4m3>);
        if (whole && a.lse) a.lse[token * a.q_heads + head] = lse2 * 0.693147180559945f;
        if (!whole) p.parts.lse2[at_part] = lse2;
      }
      const bool fix = dirty[item % kDirty] == item + 1;
      // kTiles == 1: each group writes half of the columns
      constexpr int kCols = kTiles == 1 ? kDim / 2 : kDim;
      const int col0 = kTiles == 1 ? x * kCols : 0;
#pragma unroll 1
      for (int i = col0; i < col0 + kCols; i += 32) {
        uint32_t o[32];
        tmem_ld_32cols(t_o + i, o);
        tmem_ld_wait();
        if (i + 32 == col0 + kCols) {
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_free[kTiles == 1 ? 0 : x]);
        }
        if (valid) {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * inv);
          if (whole) {
            __nv_bfloat16* dst = a.out.data + token * a.out.ts + head * a.out.hs + i;
            if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
#pragma unroll
              for (int j = 0; j < 32; j += 16) {
                uint32_t y[8];
#pragma unroll
                for (int k = 0; k < 8; ++k)
                  y[k] = f32x2_to_bf16x2(__uint_as_float(o[j + 2 * k]), __uint_as_float(o[j + 2 * k + 1]));
                st_global_32(dst + j, y);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; j += 8)
                *reinterpret_cast<uint4*>(dst + j) =
                    make_uint4(f32x2_to_bf16x2(__uint_as_float(o[j]), __uint_as_float(o[j + 1])),
                               f32x2_to_bf16x2(__uint_as_float(o[j + 2]), __uint_as_float(o[j + 3])),
                               f32x2_to_bf16x2(__uint_as_float(o[j + 4]), __uint_as_float(o[j + 5])),
                               f32x2_to_bf16x2(__uint_as_float(o[j + 6]), __uint_as_float(o[j + 7])));
            }
          } else {
            float* dst = p.parts.out + at_part * kDim + i;
#pragma unroll
            for (int j = 0; j < 32; j += 8) st_global_32(dst + j, &o[j]);
          }
        }
        __syncwarp();
      }
      if (fix && valid) {
        // values that are not finite, of the keys that not all rows see
        const int from = max(it.least(), it.key0), to = min(lim, it.key0 + count * kN);
#pragma unroll 1
        for (int key = from; key < to; ++key) {
          const int64_t page =
              checked_page(a.seqs.table[int64_t(it.s) * a.seqs.width + key / a.cache.page_size],
                           a.cache.pages, a.err);
          if (page == a.cache.pages) continue;
          const int64_t off = page * a.cache.vs[0] + key % a.cache.page_size * a.cache.vs[1] +
                              it.h * a.cache.vs[2];
#pragma unroll 1
          for (int i = col0; i < col0 + kCols; ++i) {
            const float v = kE4m3 ? e4m3_to_f32(static_cast<const uint8_t*>(a.cache.v)[off + i])
                                  : __bfloat162float(static_cast<const __nv_bfloat16*>(a.cache.v)[off + i]);
            if (isfinite(v)) continue;
            if (whole) {
              __nv_bfloat16* y = a.out.data + token * a.out.ts + head * a.out.hs + i;
              *y = __float2bfloat16_rn(__bfloat162float(*y) + v);
            } else {
              p.parts.out[at_part * kDim + i] += v;
            }
          }
        }
      }
      if (kTiles == 1) meet();                          // run_max and row_sum are free again
      __syncwarp();
      if (lane == 0) items.release(item);
    }
    if (threadIdx.x == 0) {
      note.x = flags;
      p.parts.note[blockIdx.x] = note;
    }
  } else if (warp < 12) {
    regs_dec<kHelperRegs>();
    if (warp == 9) {
      // ------------------------------------------------ MMA: O += P V
      const uint32_t id_o = idesc<kE4m3>(kDim, true);
      const uint32_t v_lo = desc_lo(smem_addr(ring), C::kVChunk);
      Place pv;
      int x = 0;                                // the score buffer (and tile)
      pv.start(items);
      VRing<C> next, at;                        // of the next block; of the one in use
      bool ok = true;
      auto ready = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && __all_sync(0xffffffffu, wait(bar, parity, abort_flag));
      };
      for (int i = 0; ok && pv.live; ++i, x ^= 1) {
        const uint32_t t_s = tmem + C::kS + x * kN;
        const uint32_t t_o = tmem + C::kO + (kTiles == 2 ? x * kDim : 0);
        const bool fresh = pv.first();
        if (kTiles == 1 || x == 0) {
          at = next;
#pragma unroll
          for (int h = 0; h < C::kPieces; ++h) next.next();
          if (!kE4m3 && lead) {
            v_slot[x] = at.slot | static_cast<int>(at.par) << 8;
            mbar_arrive(&v_known[x]);
          }
        }
        if (fresh && pv.item > 0) ready(&o_free[kTiles == 1 ? 0 : x], (pv.item - 1) & 1);
        VRing<C> r = at;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {                 // of the keys
          if ((kTiles == 1 || x == 0) && (half == 0 || C::kPieces == 2)) ready(&full[r.slot], r.par);
          ready(&p_full[2 * x + half], i >> 1 & 1);
          if (!ok) break;
          tc_fence_after_sync();
          if (lead) {
            const uint32_t v = v_lo + r.slot * (C::kSlotBytes >> 4) +
                               (C::kPieces == 2 ? 0 : half * (kN / 32) * (2048 >> 4));
            const uint32_t t_p = t_s + half * (kN / 4);
            const uint32_t acc = !fresh || half != 0;
#pragma unroll
            for (int kk = 0; kk < kN / 32; ++kk)
              umma_ts(t_o, t_p + kk * 8, v + kk * (2048 >> 4), id_o, kk == 0 ? acc : 1u);
            if ((kTiles == 1 || x == 1) && (half == 1 || C::kPieces == 2))
              umma_commit(&empty[r.slot]);
            if (half == 1) umma_commit(&pv_done[x]);
          }
          __syncwarp();
          if (C::kPieces == 2) r.next();
        }
        if (ok && (kTiles == 1 || x == 1)) {
          const int was = pv.item;
          if (pv.next(items) && lead) items.release(was);
          __syncwarp();
        }
      }
      drain();
    } else if (kE4m3 && warp == kScoreWarp) {
      score_mma();
    } else if (warp == 8 && !kE4m3) {
      copy_pages(std::false_type{});
    } else if (warp == 10 && !kE4m3) {
      copy_pages(std::true_type{});
    } else if (!kE4m3) {
      // ------------------------------------------- the schedule, and Q copies
      if (lane == 0) {
        int item = 0;
        const int rows = p.tile_tokens * a.group;
        Walk w(range, a.seqs, a.cache.heads, p.plan, a.err);
        while (publish(w, item)) {
          if (item > 0 && !wait(q_empty, (item - 1) & 1, abort_flag)) break;
          mbar_arrive_expect_tx(q_full, kTiles * (kDim / 64) * rows * 128);
          const int t0 = w.seq.q0 + w.r.tile * p.plan.tile_tokens;
#pragma unroll 1
          for (int x = 0; x < kTiles; ++x)
#pragma unroll 1
            for (int ch = 0; ch < kDim / 64; ++ch)
              tma_load_3d(q_sm + x * C::kQTile + ch * kM * 128, &tm_q, q_full, ch * 64,
                          w.r.h * a.group, t0 + x * p.tile_tokens);
          w.next(a.seqs, a.cache.heads, p.plan, a.err);
          ++item;
        }
        if (item > 0) {
          volatile int no_abort = 0;
          if (!wait(q_full, (item - 1) & 1, &no_abort)) atomicOr(a.err, NVFP4_ATTENTION_TIMEOUT);
        }
      }
      __syncwarp();
    } else if (warp == 8) {
      copy_raw(std::false_type{}, [](int) {});
    } else if (warp == 11) {
      // ------------------------------- the schedule, and the copies of V's codes
      Walk w(range, a.seqs, a.cache.heads, p.plan, a.err);
      auto ahead = [&](int item) {                  // item `item` to the other warps
        if (lane == 0) publish(w, item);
        if (w.more()) w.next(a.seqs, a.cache.heads, p.plan, a.err);
        __syncwarp();
      };
      bool all = false;                             // the end has been published
      auto more = [&](int item) {
        if (all) return;
        all = !w.more();
        ahead(item);
      };
      more(0);
      more(1);
      copy_raw(std::true_type{}, [&](int item) { more(item + 1); });
    }
  } else {
    // ------------------------------------------ K, V codes widened to f16
    if constexpr (!kE4m3) {
      regs_dec<kHelperRegs>();
      if (warp == kScoreWarp) score_mma();
    } else {
      regs_dec<kHelperRegs>();
      if (warp < 14)
        widen_pages(std::false_type{});
      else
        widen_pages(std::true_type{});
    }
  }
  if (*abort_flag && threadIdx.x == 0) atomicOr(a.err, NVFP4_ATTENTION_TIMEOUT);
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

template <int kDim, bool kE4m3, int kTiles>
int run(const Attend& a, const Device& d, cudaStream_t stream) {
  using C = Cfg<kDim, kE4m3, kTiles>;
  auto* kernel = attend_tc_kernel<kDim, kE4m3, kTiles>;
  static std::atomic<bool> ready[kMaxDevices];
  if (!ready[d.id].load(std::memory_order_acquire)) {
    // the warpgroups' shares (setmaxnreg) have to come out of what the block
    // is launched with
    cudaFuncAttributes attr;
    if (cudaFuncGetAttributes(&attr, kernel) != cudaSuccess) {
      cudaGetLastError();
      return NVFP4_ERR_LAUNCH;
    }
    constexpr int need = 256 * (kSoftmaxRegs + kHelperRegs);
    if (attr.numRegs * C::kThreads < need) return NVFP4_ERR_LAUNCH;
  }
  if (const int st = allow_smem(kernel, C::kSmem, d, ready)) return st;
  TcParams p{a, {}, Parts(a.workspace, d.num_sms, kM, kTiles, kDim), kM / a.group, 0};
  p.plan = Plan{kTiles * p.tile_tokens, kBlockShift, 1, kExtra};
  if (!countable(a.seqs, a.cache.heads, p.plan)) return NVFP4_ERR_SHAPE;
  p.box_shift = 4;
  while (p.box_shift < 7 && a.cache.page_size % (2 << p.box_shift) == 0) ++p.box_shift;
  const int box = 1 << p.box_shift;
  CUtensorMap tm_q{}, tm_k{}, tm_v{};
  if (kE4m3) {
    // rows of the units, 64 or 128 bytes of each (the readers undo the swizzle)
    constexpr int width = kDim < 128 ? 64 : 128;
    using UV = Units<C, kDim, true>;
    if (!page_map(&tm_k, a.cache, false, width, std::min(box, Units<C, kDim, false>::kRows), 1) ||
        !page_map(&tm_v, a.cache, true, width, std::min(box, UV::kRows), box >= UV::kRows ? UV::kChunks : 1))
      return NVFP4_ERR_LAUNCH;
  } else if (!query_map(&tm_q, a.q, a.cache.dim, a.q_heads, a.seqs.tokens, a.group, p.tile_tokens) ||
             !page_map(&tm_k, a.cache, false, 64, box, 1) ||
             !page_map(&tm_v, a.cache, true, 64, std::min(box, C::kVKeys),
                       box >= C::kVKeys ? C::kVChunks : 1)) {
    return NVFP4_ERR_LAUNCH;
  }
  if (const int st = launch(kernel, dim3(d.num_sms), dim3(C::kThreads), C::kSmem, stream, tm_q, tm_k,
                            tm_v, p))
    return st;
  return run_join(int64_t(a.max_q_len) * a.group > kM, a, p.parts, p.plan, d.num_sms, d.id, stream);
}

// One tile of rows; more: two tiles in a CTA, where TMEM has room for two
// accumulators.
template <int kDim, bool kE4m3>
int run_tiles(bool two, const Attend& a, const Device& d, cudaStream_t stream) {
  if constexpr (kDim < 256)
    if (two) return run<kDim, kE4m3, 2>(a, d, stream);
  return run<kDim, kE4m3, 1>(a, d, stream);
}

}  // namespace

int64_t attend_tc_workspace(int head_dim, const Device& d) {
  return Parts::bytes(d.num_sms, 2 * kM, head_dim);
}

int run_attend_tc(int64_t rows, const Attend& a, const Device& d, cudaStream_t stream) {
  const bool two = rows > kM, f8 = a.cache.e4m3;
  switch (a.cache.dim) {
    case 64:
      return f8 ? run_tiles<64, true>(two, a, d, stream) : run_tiles<64, false>(two, a, d, stream);
    case 128:
      return f8 ? run_tiles<128, true>(two, a, d, stream) : run_tiles<128, false>(two, a, d, stream);
    default:
      return f8 ? run_tiles<256, true>(two, a, d, stream) : run_tiles<256, false>(two, a, d, stream);
  }
}

}  // namespace attn
}  // namespace nvfp4
