// The attention kernel behind packed cross attention and attention over a paged cache (TMA + tcgen05 + TMEM), over a
// Source that says what an item is, where its tiles come from and what a row sees, and the kernel that joins the
// chunks of cut items.  Its structure and what it measured stand in cross_attn_sm103.cu.
//
// A Source is a kernel parameter with
//   kDim, kChunks (of an item, at most), kConvert (tiles arrive as bytes and are converted by the epilogue's warps),
//     kRowLimits (rows of a tile see unlike numbers of keys);  tmap_q, tmap_k, tmap_v;  seg;  q_bytes() of a query tile
//   Work: an item -- ntiles (0: no more work), q0[2] (first row of each tile), seg_end, q_head(t), nkv and last_keys
//     (key tiles, and keys in the last of them; 0 for none), partial (entry whose partial results the item
//     writes, -1 for o itself)
//   Entry: an entry of the last wave, with chunks (1: a whole item)
//   whole_item(k): a CTA's k-th whole item;  decode(item, ws, split_area): its Work;  place(entry, t): a tile's place
//   row(r): token and head of a tile's row r;  row_keys(work, t, row): keys it sees from the item's first one on
//   Fetch: the key/value producer's state;  convert_row: a row of bytes into a bf16 tile
#pragma once

#include <cuda_bf16.h>

#include "h3_internal.h"
#include "launch.h"
#include "sm103_ptx.cuh"

namespace h3 {
namespace {

constexpr int kBlockM = 128, kBlockN = 128;
constexpr int kTileThreads = 512;
constexpr int kRegsSoftmax = 176, kRegsEpilogue = 80, kRegsOther = 80;
static_assert(2 * kRegsSoftmax + kRegsEpilogue + kRegsOther == 65536 / 128, "the split of the registers at launch");
constexpr int kTmemCols = 512, kColO = 0, kColS = 256;
constexpr float kRescaleLog2 = 8.0f;  // rescale O only when the running max grows by > 2^8
constexpr int kHeader = kAttnWsHeaderWords;

__host__ __device__ constexpr int key_tiles(int keys) {
  return keys > 0 ? (keys + kBlockN - 1) / kBlockN : 1;
}

// The split area: entries (a chunk of the last wave, or a whole item of it), then the first entries of the cut items
// (fewer than a wave), the first entry of each CTA and their number, then the partial results.
template <typename Entry>
__host__ __device__ constexpr size_t split_items_offset() {
  return static_cast<size_t>(kSplitMaxEntries) * sizeof(Entry);
}
template <typename Entry>
__host__ __device__ constexpr size_t split_partials_offset() {
  return split_items_offset<Entry>() + static_cast<size_t>(kSplitMaxEntries) * sizeof(uint32_t);
}
template <int D>
constexpr size_t kPartial = static_cast<size_t>(kBlockM) * (D + 1);  // floats of a tile's partial

struct TileRow {
  int token, head;  // past the tile's first row and head; a row that is none has a token past every segment
};
struct TilePlace {
  bool exists;
  int q0, head, seg_end;
};

template <typename T>
__device__ __forceinline__ T block_exclusive_scan(T v, T* s_warp, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  T before = 0, all = 0;
#pragma unroll 1
  for (int w = 0; w < static_cast<int>(blockDim.x) / 32; ++w) {
    if (w < warp) before += s_warp[w];
    all += s_warp[w];
  }
  total = all;
  return before + x - v;
}

template <typename Source>
struct TileCfg {
  static constexpr int D = Source::kDim;
  static constexpr int kBoxes = D / 64;
  static constexpr int kTileBytes = kBlockM * D * 2;
  static constexpr int kBoxBytes = kBlockM * 128;
  // key and value tiles in turn; with tiles that arrive as bytes, a ring of those before it
  static constexpr int kRawBytes = kBlockN * D;  // the rows' scales, a byte each, lie behind the ring
  static constexpr int kRaws = Source::kConvert ? (D == 128 ? 2 : 4) : 0;
  static constexpr int kStages = Source::kConvert ? (D == 128 ? 4 : 8) : (D == 128 ? 5 : 8);
  // q_full[2], q_empty[2], s_full[2], p_half[2], p_full[2], o_final[2], o_empty[2], l_full[2],
  // w_full[2], w_empty[2], drain[2], turn[2], then kv_full, kv_empty, v_tail, raw_full, raw_empty
  static constexpr int kNumBars = 24 + 3 * kStages + 2 * kRaws;
  static constexpr int kSmemBytes = 1024 + kTileBytes * (2 + kStages) + kRaws * (kRawBytes + kBlockN) + kNumBars * 8 + 24 +
                                    2 * sizeof(typename Source::Work) + 2 * kBlockM * sizeof(float);
  static_assert(kSmemBytes <= 232448, "shared memory of one CTA");
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(kBlockM, kBlockN, false);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(kBlockM, D, true);
};

template <typename Source>
__global__ void __launch_bounds__(kTileThreads, 1)
attn_tile_kernel(const __grid_constant__ Source src, __nv_bfloat16* __restrict__ out, int wide, float* __restrict__ lse,
                 float scale, float scale_log2, const uint32_t* __restrict__ ws, uint8_t* __restrict__ split_area,
                 unsigned int* err, unsigned long long wait_ns, unsigned int stall_after) {
  using C = TileCfg<Source>;
  using Work = typename Source::Work;
  using Entry = typename Source::Entry;
  constexpr int D = Source::kDim;
  constexpr int kStages = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = sQ + 2 * C::kTileBytes;
  uint8_t* sRaw = sKV + kStages * C::kTileBytes;
  uint8_t* sScale = sRaw + C::kRaws * C::kRawBytes;
  float* s_norm = reinterpret_cast<float*>(sScale + C::kRaws * kBlockN);  // [2][128]: 1 / row sum
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_norm + 2 * kBlockM);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::kNumBars);
  Work* work = reinterpret_cast<Work*>(tmem_slot + 2);  // 2-slot ring
  const uint32_t bar0 = smem_u32(bars);
  auto bar = [&](int i) { return bar0 + 8 * static_cast<uint32_t>(i); };
  auto bar_qfull = [&](int t) { return bar(t); };
  auto bar_qempty = [&](int t) { return bar(2 + t); };
  auto bar_sfull = [&](int t) { return bar(4 + t); };
  auto bar_phalf = [&](int t) { return bar(6 + t); };
  auto bar_pfull = [&](int t) { return bar(8 + t); };
  auto bar_ofinal = [&](int t) { return bar(10 + t); };
  auto bar_oempty = [&](int t) { return bar(12 + t); };
  auto bar_lfull = [&](int t) { return bar(14 + t); };
  auto bar_wfull = [&](int i) { return bar(16 + i); };
  auto bar_wempty = [&](int i) { return bar(18 + i); };
  auto bar_drain = [&](int t) { return bar(20 + t); };
  auto bar_turn = [&](int t) { return bar(22 + t); };
  auto bar_full = [&](int s) { return bar(24 + s); };
  auto bar_empty = [&](int s) { return bar(24 + kStages + s); };
  auto bar_vtail = [&](int s) { return bar(24 + 2 * kStages + s); };
  auto bar_rfull = [&](int i) { return bar(24 + 3 * kStages + i); };
  auto bar_rempty = [&](int i) { return bar(24 + 3 * kStages + C::kRaws + i); };

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto pwait = [&](uint32_t b, uint32_t parity) { return mbar_wait(b, parity, wait_ns); };
  // The whole warp polls: a branch for one lane would leave the warp diverged behind it.
  auto wait_all = [&](uint32_t b, uint32_t parity) { return __all_sync(0xffffffffu, pwait(b, parity)) != 0; };
  auto wait_long = [&](uint32_t b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_long(b, parity, wait_ns)) != 0;
  };
  // One arrival for the warp, after what all its lanes did.
  auto arrive_warp = [&](uint32_t b) {
    __syncwarp();
    if (lane == 0) mbar_arrive(b);
  };

  // set up while the plan is made: nothing of it is read before the wait
  if (warp == 12 && lane == 0) {
    tma_prefetch_desc(&src.tmap_q);
    tma_prefetch_desc(&src.tmap_k);
    tma_prefetch_desc(&src.tmap_v);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar_qfull(t), 1);
      mbar_init(bar_qempty(t), 1);
      mbar_init(bar_sfull(t), 1);
      mbar_init(bar_phalf(t), 4);  // warps
      mbar_init(bar_pfull(t), 4);  // warps
      mbar_init(bar_ofinal(t), 1);
      mbar_init(bar_oempty(t), 4);  // warps
      mbar_init(bar_lfull(t), 4);  // warps
      mbar_init(bar_wfull(t), 1);
      mbar_init(bar_drain(t), 1);
      mbar_init(bar_turn(t), 1);
      mbar_init(bar_wempty(t), 15);  // softmax and epilogue warps, key/value producer, MMA warps
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(bar_full(s), Source::kConvert ? 4 : 1);  // the copy, or the warps that convert
      mbar_init(bar_empty(s), 2);  // MMA warps
      mbar_init(bar_vtail(s), 1);
    }
    for (int i = 0; i < C::kRaws; ++i) {
      mbar_init(bar_rfull(i), 1);
      mbar_init(bar_rempty(i), 4);  // warps that convert
    }
    fence_mbarrier_init();
  }
  if (warp == 13) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_dependency_wait();
  launch_dependents();
  // this CTA's items: every gridDim.x-th of the whole ones, then its entries of the last wave
  const uint32_t whole = ws[2];  // of all CTAs
  uint32_t entry = 0, entry_end = 0;
  if (split_area != nullptr) {  // (read before it is known whether there are any)
    const uint32_t* firsts = reinterpret_cast<const uint32_t*>(split_area + split_items_offset<Entry>()) + gridDim.x;
    entry = firsts[blockIdx.x];
    entry_end = firsts[blockIdx.x + 1];
  }
  if (ws[3] == 0) entry = entry_end = 0;
  // nothing to do, or a timeout recorded earlier and not read yet: leave at once, all threads together
  const bool late = err != nullptr && *reinterpret_cast<volatile unsigned int*>(err) == kErrTimeout;
  if (__syncthreads_or(late) || (blockIdx.x >= whole && entry == entry_end)) {
    if (warp == 13) tmem_dealloc(tmem, kTmemCols);
    return;
  }

  // Item k from the ring, for one warp (every lane calls).  False when the wait ran out.
  auto take = [&](int k, Work& d) {
    if (!wait_long(bar_wfull(k & 1), (k >> 1) & 1)) return false;
    d = work[k & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_wempty(k & 1));
    return true;
  };

  // An item's last key tile is multiplied as far as it holds keys, in steps of 16 and at least one; value
  // rows past the keys that PV reads all the same are zeroed.
  auto steps16 = [](int keys) { return max(1, (keys + 15) / 16); };
  // (what converts a tile zeroes them as it writes it)
  auto has_tail = [&](int keys) { return !Source::kConvert && keys < 16 * steps16(keys); };

  if (warp >= 12) {
    setmaxnreg_dec<kRegsOther>();
    if (warp == 12) {
      // ================= key/value producer =================
      const uint64_t pol_keep = l2_policy_evict_last();  // shared by the CTAs of a key head
      uint32_t loaded = 0, v_last = 0;  // tiles; the last value tile of an item
      int tail_keys = 0;
      bool ok = true, stalled = false, tail = false;
      Work d;
      // The tail of an item's last value tile, once it has landed: while the next key tile is on its way,
      // before the next value tile.  (Whole 128-byte rows: the swizzle permutes 16-byte pieces within a row.)
      auto zero_tail = [&] {
        if (!tail) return true;
        tail = false;
        const uint32_t s = v_last % kStages;
        if (!wait_long(bar_full(s), (v_last / kStages) & 1)) return false;
        uint8_t* vb = sKV + s * C::kTileBytes;
        for (int i = lane; i < (16 * steps16(tail_keys) - tail_keys) * C::kBoxes * 8; i += 32) {
          const int r = tail_keys + i / (C::kBoxes * 8), rem = i % (C::kBoxes * 8);
          *reinterpret_cast<uint4*>(vb + (rem >> 3) * C::kBoxBytes + r * 128 + (rem & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        arrive_warp(bar_vtail(s));
        return true;
      };
      for (int k = 0; ok && !stalled; ++k) {
        ok = take(k, d);
        if (!ok || d.ntiles == 0) break;
        typename Source::Fetch fetch(src, d);
        for (int j = 0; j < d.nkv; ++j) {
          if (loaded / 2 >= stall_after) {  // testing hook: as if the loads had stalled
            stalled = true;
            break;
          }
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            if constexpr (Source::kConvert) {
              const int i = static_cast<int>(loaded % C::kRaws);
              ok = wait_long(bar_rempty(i), ((loaded / C::kRaws) & 1) ^ 1);
              if (!ok) break;
              fetch.tile(src, d, j, v, sRaw + i * C::kRawBytes, sScale + i * kBlockN, bar_rfull(i), pol_keep, err);
            } else {
              const int s = static_cast<int>(loaded % kStages);
              ok = (v == 0 || zero_tail()) && wait_long(bar_empty(s), ((loaded / kStages) & 1) ^ 1);
              if (!ok) break;
              fetch.tile(src, d, j, v, sKV + s * C::kTileBytes, nullptr, bar_full(s), pol_keep, err);
            }
            ++loaded;
          }
          if (!ok) break;
        }
        tail = ok && !stalled && has_tail(d.last_keys);
        tail_keys = d.last_keys;
        v_last = loaded - 1;
      }
      if (ok && !stalled) ok = zero_tail();
      if (!ok && lane == 0) record_error(err, kErrTimeout);
      // never leave while a copy may still land: the last loads sit on distinct stages
      constexpr uint32_t kRing = Source::kConvert ? C::kRaws : kStages;
      for (uint32_t i = 0; i < kRing && i < loaded; ++i) {
        const uint32_t n = loaded - 1 - i;
        mbar_wait(Source::kConvert ? bar_rfull(n % kRing) : bar_full(n % kRing), (n / kRing) & 1);
      }
    } else if (warp == 15) {
      // ================= scheduler and query producer =================
      const uint64_t pol_stream = l2_policy_evict_first();
      uint32_t qn[2] = {0u, 0u};
      bool ok = true;
      for (int k = 0; ok; ++k) {
        const uint32_t item = Source::whole_item(static_cast<uint32_t>(k));
        Work d{};
        if (item < whole) d = src.decode(item, ws, split_area);
        else if (entry < entry_end) d = src.decode(whole + entry++, ws, split_area);
        ok = wait_long(bar_wempty(k & 1), ((k >> 1) & 1) ^ 1);
        if (!ok) break;
        if (lane == 0) {
          work[k & 1] = d;
          mbar_arrive(bar_wfull(k & 1));
        }
        __syncwarp();
        if (d.ntiles == 0) break;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (t >= d.ntiles) break;
          ok = wait_long(bar_qempty(t), (qn[t] & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar_qfull(t), src.q_bytes());
            for (int x = 0; x < C::kBoxes; ++x)
              tma_load_3d_hint(smem_u32(sQ + t * C::kTileBytes + x * C::kBoxBytes), &src.tmap_q, x * 64, d.q_head(t),
                               d.q0[t], bar_qfull(t), pol_stream);
          }
          ++qn[t];
        }
      }
      if (!ok && lane == 0) record_error(err, kErrTimeout);
      for (int t = 0; t < 2; ++t)
        if (qn[t] > 0) mbar_wait(bar_qfull(t), (qn[t] - 1) & 1);
    } else {
      // ================= MMA issuers: warp 13 for tile 0, 14 for tile 1 =================
      // A warp's polls wait for the products that it has issued before, so the tensor core would run dry at
      // each poll of a single issuer.  Two take turns: what one polls for, it does while the other's products
      // run.  Their order is kept (a turn barrier each), or the tiles would fall in phase.
      const int t = warp - 13;
      constexpr uint32_t kTile16 = C::kTileBytes >> 4;
      const SmemDesc dq = sw128_desc_split(smem_u32(sQ) + t * C::kTileBytes, 16, 1024);
      const SmemDesc dk = sw128_desc_split(smem_u32(sKV), 16, 1024);
      const SmemDesc dv = sw128_desc_split(smem_u32(sKV), C::kBoxBytes, 1024);
      const uint32_t s_tmem = tmem + kColS + 128 * t, o_tmem = tmem + kColO + 128 * t;
      auto issue_qk = [&](int s, uint32_t idesc) {  // S_t = Q_t K_s^T
        const uint32_t klo = dk.lo + s * kTile16;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
          mma_ss_split(s_tmem, dq.lo + off, dq.hi, klo + off, dk.hi, idesc, kk > 0 ? 1u : 0u);
        }
        mma_commit(bar_sfull(t));
      };
      auto issue_pv = [&](int s, bool first, int from) {  // O_t += P_t V_s over four steps of 16 keys
        const uint32_t vlo = dv.lo + s * kTile16;
#pragma unroll
        for (int kk = from; kk < from + 4; ++kk)
          mma_ts_split(o_tmem, s_tmem + kk * 8, vlo + kk * (2048 >> 4), dv.hi, C::kIdescPV,
                       (!first || kk > 0) ? 1u : 0u);
      };
      const bool leader = elect_one();
      struct Item {  // what is needed of an item here
        int ntiles, nkv, last_keys;
      } cur{0, 0, 0}, nxt{0, 0, 0};
      auto take_item = [&](int k, Item& i) {
        if (!wait_all(bar_wfull(k & 1), (k >> 1) & 1)) return false;
        i = Item{work[k & 1].ntiles, work[k & 1].nkv, work[k & 1].last_keys};
        __syncwarp();
        if (leader) mbar_arrive(bar_wempty(k & 1));
        return true;
      };
      auto idesc_last = [&](const Item& i) {
        return i.last_keys < kBlockN ? idesc_bf16_f32(kBlockM, 16 * steps16(i.last_keys), false) : C::kIdescQK;
      };
      int sk = 0, sv = 1;
      uint32_t pk = 0, pv = 0;  // phases of the stages of the next key and value tile
      uint32_t qp = 0u, pp = 0u, op = 1u, turn = t == 0 ? 1u : 0u;  // phases of Q, P, O and the turns
      uint32_t tails = 0;  // phases of the value tails, a bit per stage
      auto next_k = [&] {
        if ((sk += 2) >= kStages) {
          sk -= kStages;
          pk ^= 1;
        }
      };
      auto next_v = [&] {
        if ((sv += 2) >= kStages) {
          sv -= kStages;
          pv ^= 1;
        }
      };
      // Waits for this warp's turn and whatever else is asked for; the polls overlap.
      auto wait_turn = [&](bool v, bool k, bool q, bool p, uint32_t p_bar, bool o, bool z) {
        bool r[7];
        r[0] = !p || mbar_try_wait(p_bar, pp);
        r[1] = mbar_try_wait(bar_turn(t), turn);
        r[2] = !v || mbar_try_wait(bar_full(sv), pv);
        r[3] = !k || mbar_try_wait(bar_full(sk), pk);
        r[4] = !q || mbar_try_wait(bar_qfull(t), qp);
        r[5] = !o || mbar_try_wait(bar_oempty(t), op);
        r[6] = !z || mbar_try_wait(bar_vtail(sv), tails >> sv & 1u);
        bool all = true;
        if (!r[0]) all = pwait(p_bar, pp);
        if (!r[1]) all = pwait(bar_turn(t), turn) && all;
        if (!r[2]) all = pwait(bar_full(sv), pv) && all;
        if (!r[3]) all = pwait(bar_full(sk), pk) && all;
        if (!r[4]) all = pwait(bar_qfull(t), qp) && all;
        if (!r[5]) all = pwait(bar_oempty(t), op) && all;
        if (!r[6]) all = pwait(bar_vtail(sv), tails >> sv & 1u) && all;
        turn ^= 1;
        if (z) tails ^= 1u << sv;
        if (q) qp ^= 1;
        if (o) op ^= 1;
        return __all_sync(0xffffffffu, all) != 0;
      };
      bool ok = take_item(0, cur), issued = false;
      if (ok && cur.ntiles > 0) {  // the first item's first scores
        ok = wait_all(bar_full(0), 0);
        if (ok && t < cur.ntiles) {
          ok = wait_all(bar_qfull(t), 0);
          qp = 1;
          tc_fence_after();
          if (ok && leader) {
            issue_qk(0, cur.nkv == 1 ? idesc_last(cur) : C::kIdescQK);
            if (cur.nkv == 1) mma_commit(bar_qempty(t));
            mma_commit(bar_empty(0));
          }
          issued = ok;
          __syncwarp();
        } else if (ok && leader) {
          mbar_arrive(bar_empty(0));
        }
        next_k();
      }
      // One step within an item: PV of its key tile, and the scores of the next one.
      auto step = [&](bool first, uint32_t idesc, bool q_done) {
        if (t < cur.ntiles) {
          if (!wait_turn(true, true, false, true, bar_phalf(t), first, false)) return false;
          tc_fence_after();
          if (leader) issue_pv(sv, first, 0);
          __syncwarp();
          if (!wait_all(bar_pfull(t), pp)) return false;
          pp ^= 1;
          tc_fence_after();
          if (leader) issue_pv(sv, false, 4);
          if (leader) {
            mma_commit(bar_empty(sv));
            issue_qk(sk, idesc);
            if (q_done) mma_commit(bar_qempty(t));
            mma_commit(bar_empty(sk));
            mbar_arrive(bar_turn(t ^ 1));
          }
          __syncwarp();
        } else {
          if (!wait_turn(true, true, false, false, 0, false, false)) return false;
          if (leader) {
            mbar_arrive(bar_empty(sv));
            mbar_arrive(bar_empty(sk));
            mbar_arrive(bar_turn(t ^ 1));
          }
          __syncwarp();
        }
        next_v();
        next_k();
        return true;
      };
      // The step between two items: PV of the last key tile, as far as it holds keys, and the next item's
      // first scores.
      auto boundary = [&](bool first) {
        const bool has_pv = t < cur.ntiles, has_qk = t < nxt.ntiles, more = nxt.ntiles > 0;
        const int end = steps16(cur.last_keys);
        const uint32_t idesc = nxt.nkv == 1 ? idesc_last(nxt) : C::kIdescQK;
        if (!wait_turn(true, more, has_qk, has_pv, bar_pfull(t), has_pv && first,
                       has_tail(cur.last_keys))) return false;
        if (has_pv) pp ^= 1;
        tc_fence_after();
        if (has_pv) {
          if (end == kBlockN / 16) {
            if (leader) {
              issue_pv(sv, first, 0);
              issue_pv(sv, false, 4);
            }
          } else if (leader) {
#pragma unroll 1
            for (int kk = 0; kk < end; ++kk)
              mma_ts_split(o_tmem, s_tmem + kk * 8, dv.lo + sv * kTile16 + kk * (2048 >> 4), dv.hi, C::kIdescPV,
                           (!first || kk > 0) ? 1u : 0u);
          }
          if (leader) {
            mma_commit(bar_ofinal(t));
            mma_commit(bar_empty(sv));
          }
        } else if (leader) {
          mbar_arrive(bar_empty(sv));
        }
        __syncwarp();
        if (has_qk) {
          if (leader) {
            issue_qk(sk, idesc);
            if (nxt.nkv == 1) mma_commit(bar_qempty(t));
            mma_commit(bar_empty(sk));
          }
          issued = true;
        } else if (more && leader) {
          mbar_arrive(bar_empty(sk));
        }
        __syncwarp();
        if (leader) mbar_arrive(bar_turn(t ^ 1));
        __syncwarp();
        next_v();
        if (more) next_k();
        return true;
      };
      for (int k = 0; ok && cur.ntiles > 0; ++k) {
        const uint32_t idesc_end = idesc_last(cur);
        for (int j = 0; j + 1 < cur.nkv && ok; ++j) {
          const bool q_done = j + 2 == cur.nkv;
          ok = step(j == 0, q_done ? idesc_end : C::kIdescQK, q_done);
        }
        if (ok) ok = take_item(k + 1, nxt);
        if (ok) ok = boundary(cur.nkv == 1);
        cur = nxt;
      }
      if (!ok && leader) record_error(err, kErrTimeout);
      if (issued && leader) {  // every MMA issued has completed before TMEM is released
        mma_commit(bar_drain(t));
        mbar_wait(bar_drain(t), 0);
      }
      __syncwarp();
    }
  } else if (warp >= 8) {
    setmaxnreg_dec<kRegsEpilogue>();
    // ================= epilogue: O / l -> bf16 rows (or fp32 partials) =================
    const int row = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t fn[2] = {0u, 0u};
    bool ok = true;
    const int odd = lane & 1;
    const TileRow even = src.row(row - odd), next = src.row(row - odd + 1);
    auto finish = [&](const Work& d) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (t >= d.ntiles) break;
      const bool there = wait_long(bar_lfull(t), fn[t] & 1) && wait_long(bar_ofinal(t), fn[t] & 1);
      ++fn[t];
      if (!there) return false;
      tc_fence_after();
      const float inv_l = s_norm[t * kBlockM + row];
      const uint32_t o_addr = tmem + lane_base + kColO + 128 * t;
      if (d.partial >= 0) {
        float* mine = reinterpret_cast<float*>(split_area + split_partials_offset<Entry>()) +
                      (static_cast<size_t>(d.partial) * 2 + t) * kPartial<D> + static_cast<size_t>(row) * D;
        const bool sectors = (reinterpret_cast<uintptr_t>(mine) & 31u) == 0;
        const bool real = d.q0[t] + (odd ? next : even).token < d.seg_end;  // this thread's row is one
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t r[32];
          tmem_ld32(o_addr + c0, r);
          tmem_ld_wait();
          tmem_reg_fence<32>(r);
#pragma unroll
          for (int c = 0; c < 32; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * inv_l);
#pragma unroll
          for (int c = 0; c < 32; c += 8)
            if (real) st_global_32(mine + c0 + c, r + c, sectors);
        }
        tc_fence_before();
        arrive_warp(bar_oempty(t));
        continue;
      }
      // Lanes 2i and 2i + 1 trade halves of each 64 bytes, so that an instruction writes whole
      // 32-byte sectors, two neighbours of a row at a time.
      const int r0 = d.q0[t] + even.token, r1 = d.q0[t] + next.token;  // the even lane's row and the one behind
      __nv_bfloat16* p0 = out + (static_cast<size_t>(r0) * src.seg.num_q_heads + d.q_head(t) + even.head) * D + 16 * odd;
      __nv_bfloat16* p1 = out + (static_cast<size_t>(r1) * src.seg.num_q_heads + d.q_head(t) + next.head) * D + 16 * odd;
#pragma unroll 1
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t r[32], pk[16];
        tmem_ld32(o_addr + c0, r);
        tmem_ld_wait();
        tmem_reg_fence<32>(r);
        if (c0 == D - 32) {
          tc_fence_before();
          arrive_warp(bar_oempty(t));
        }
#pragma unroll
        for (int c = 0; c < 16; ++c)
          pk[c] = pack_bf16x2(__uint_as_float(r[2 * c]) * inv_l, __uint_as_float(r[2 * c + 1]) * inv_l);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? pk[c] : pk[8 + c], 1);
          pk[c] = odd ? got : pk[c];
          pk[8 + c] = odd ? pk[8 + c] : got;
        }
        if (r0 < d.seg_end) st_global_32(p0 + c0, pk, wide);
        if (r1 < d.seg_end) st_global_32(p1 + c0, pk + 8, wide);
      }
    }
      return true;
    };
    if constexpr (!Source::kConvert) {
      Work d;
      for (int k = 0; ok; ++k) {
        ok = take(k, d);
        if (!ok || d.ntiles == 0) break;
        ok = finish(d);
      }
    } else {
      // These warps also turn the tiles, which arrive as bytes, into bf16: row r of a tile is thread r's.  An
      // item's O is read out behind the next item's first two tiles, so that its products have those.
      uint32_t cn = 0;  // tiles
      auto convert = [&](const Work& d, int j, bool v) {
        const uint32_t i = cn % C::kRaws, s = cn % kStages;
        if (!wait_long(bar_rfull(i), (cn / C::kRaws) & 1) || !wait_long(bar_empty(s), ((cn / kStages) & 1) ^ 1)) return false;
        ++cn;
        const int keys = j == d.nkv - 1 ? d.last_keys : kBlockN;
        Source::convert_row(sRaw + i * C::kRawBytes, sScale[i * kBlockN + row], sKV + s * C::kTileBytes, row, row < keys,
                            v && row < 16 * steps16(keys));
        fence_proxy_async_smem();
        arrive_warp(bar_full(s));
        arrive_warp(bar_rempty(i));
        return true;
      };
      Work d[2];
      for (int k = 0; ok; ++k) {
        Work& cur = d[0];
        ok = take(k, cur);
        if (!ok) break;
        for (int j = 0; ok && cur.ntiles > 0 && j < cur.nkv; ++j) {
          ok = convert(cur, j, false) && convert(cur, j, true);
          if (ok && j == 0 && k > 0) ok = finish(d[1]);
        }
        if (!ok) break;
        if (cur.ntiles == 0) {
          if (k > 0) ok = finish(d[1]);
          break;
        }
        d[1] = cur;
      }
    }
    if (!ok && lane == 0) record_error(err, kErrTimeout);
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ================= softmax (warps 0-3: tile 0, 4-7: tile 1) =================
    const int t = warp >> 2;
    const int row = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_base + kColS + 128 * t;
    const uint32_t o_addr = tmem + lane_base + kColO + 128 * t;
    const float2 c2 = make_float2(scale_log2, scale_log2);
    const TileRow mine = src.row(row);
    uint32_t sn = 0, un = 0;  // score tiles and items of this query tile seen
    bool ok = true;
    Work d;
    for (int k = 0; ok; ++k) {
      ok = take(k, d);
      if (!ok || d.ntiles == 0) break;
      if (t >= d.ntiles) continue;
      const int row_keys = src.row_keys(d, t, mine);  // of the item's, that this row sees
      float m_used = -INFINITY, l = 0.f;
      // New row max: the reference max moves (and l and O_t are rescaled) only when it grows by more
      // than 2^kRescaleLog2.  O_t is stable here: PV_t,{j-1} was issued before the scores whose
      // completion this thread has seen.
      auto update_max = [&](float mx, int j) {
        float alpha = 1.f;
        bool rescale = false;
        if (mx > m_used && (m_used == -INFINITY || (mx - m_used) * scale_log2 > kRescaleLog2)) {
          alpha = ex2_approx((m_used - mx) * scale_log2);
          rescale = j > 0;
          l *= alpha;
          m_used = mx;
        }
        if (__any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t r[32];
            tmem_ld32(o_addr + c0, r);
            tmem_ld_wait();
            tmem_reg_fence<32>(r);
#pragma unroll
            for (int c = 0; c < 32; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * alpha);
            tmem_st32(o_addr + c0, r);
          }
        }
        // a row without keys has no max: its weights are exp2(-inf) = 0
        const float mb = m_used == -INFINITY ? 0.f : m_used * scale_log2;
        return make_float2(-mb, -mb);
      };
      // weights of 64 scores as 32 packed bf16 pairs; acc: four running sums
      auto weights = [&](const uint32_t* s, float2 nm2, float2 (&acc)[4], uint32_t* p) {
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float2 x = ffma2(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), c2, nm2);
          const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
          acc[c & 3] = fadd2(acc[c & 3], e);
          p[c] = pack_bf16x2(e.x, e.y);
        }
      };
      for (int j = 0; j < d.nkv; ++j) {
        ok = wait_all(bar_sfull(t), sn++ & 1);
        if (!ok) break;
        tc_fence_after();
        const int keys = j == d.nkv - 1 ? d.last_keys : kBlockN;
        const int seen = Source::kRowLimits ? min(keys, row_keys - j * kBlockN) : keys;
        float2 acc[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        // row max of columns: four chains of 3-input steps
        auto max_of = [&](const uint32_t* s, int n) {
#pragma unroll
          for (int c = 0; c < n; c += 8)
#pragma unroll
            for (int u = 0; u < 4; ++u)
              m4[u] = fmax3(m4[u], __uint_as_float(s[c + u]), __uint_as_float(s[c + 4 + u]));
          return fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        };
        uint32_t s[128], p[32];
        tmem_ld32(s_addr, s);
        tmem_ld32(s_addr + 32, s + 32);
        if (keys <= 64) {  // a short last tile: half the columns
          tmem_ld_wait();
          tmem_reg_fence<64>(s);
#pragma unroll
          for (int c = 0; c < 64; ++c) s[c] = c < seen ? s[c] : 0xff800000u;
          weights(s, update_max(max_of(s, 64), j), acc, p);
          tmem_st32(s_addr, p);
          tmem_st_wait();
          tc_fence_before();
          arrive_warp(bar_phalf(t));
        } else {
          tmem_ld32(s_addr + 64, s + 64);
          tmem_ld32(s_addr + 96, s + 96);
          tmem_ld_wait();
          tmem_reg_fence<128>(s);
          if constexpr (Source::kRowLimits) {
            if (__any_sync(0xffffffffu, seen < kBlockN)) {
#pragma unroll
              for (int c = 0; c < 128; ++c) s[c] = c < seen ? s[c] : 0xff800000u;
            }
          } else if (keys < kBlockN) {  // keys past the end: by select, so NaN/Inf there is discarded
#pragma unroll
            for (int c = 64; c < 128; ++c) s[c] = c < keys ? s[c] : 0xff800000u;
          }
          const float2 nm2 = update_max(max_of(s, 128), j);
          weights(s, nm2, acc, p);
          tmem_st32(s_addr, p);
          tmem_st_wait();
          tc_fence_before();
          arrive_warp(bar_phalf(t));
          weights(s + 64, nm2, acc, p);
          tmem_st32(s_addr + 32, p);
          tmem_st_wait();
          tc_fence_before();
        }
        arrive_warp(bar_pfull(t));
        const float2 a01 = fadd2(acc[0], acc[1]), a23 = fadd2(acc[2], acc[3]);
        l += (a01.x + a01.y) + (a23.x + a23.y);
      }
      if (!ok) break;
      // hand the row's norm to the epilogue, once it has read the previous item's
      if (un > 0) ok = wait_all(bar_oempty(t), (un - 1) & 1);
      if (!ok) break;
      ++un;
      s_norm[t * kBlockM + row] = l == 0.f ? 0.f : 1.f / l;
      arrive_warp(bar_lfull(t));
      const float lse_row = m_used * scale + logf(l);  // -inf without keys
      const int q_row = d.q0[t] + mine.token;
      if (d.partial >= 0)
        (reinterpret_cast<float*>(split_area + split_partials_offset<Entry>()) +
         (static_cast<size_t>(d.partial) * 2 + t) * kPartial<D>)[static_cast<size_t>(kBlockM) * D + row] = lse_row;
      else if (lse != nullptr && q_row < d.seg_end)
        lse[static_cast<size_t>(d.q_head(t) + mine.head) * src.seg.capacity_q + q_row] = lse_row;
    }
    if (!ok && lane == 0) record_error(err, kErrTimeout);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Merge of cut items, in chunk order: lse = log sum_c exp(lse_c), o = sum_c exp(lse_c - lse) o_c.
// A unit is 16 rows of one tile; memory-bound and short (the partials are in L2).
struct Float8 {
  float4 x, y;
};
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = 16;
static_assert(kMergeThreads == 16 * kMergeRows, "16 lanes to a row");
constexpr int kMergeUnits = 2 * (kBlockM / kMergeRows);
template <typename Source>
__global__ void __launch_bounds__(kMergeThreads)
attn_tile_merge_kernel(const uint32_t* __restrict__ ws, const uint8_t* __restrict__ split_area,
                       __nv_bfloat16* __restrict__ out, float* __restrict__ lse, const __grid_constant__ Source src,
                       const unsigned int* err) {
  constexpr int D = Source::kDim;
  using Entry = typename Source::Entry;
  __shared__ float s_w[kMergeRows][Source::kChunks];
  grid_dependency_wait();
  launch_dependents();
  // What is read here comes one read after another, each some 0.7 us: so the first item is read before it is known to
  // be one, and a thread's values of the first chunks with the chunks' LSEs.
  const uint32_t* items = reinterpret_cast<const uint32_t*>(split_area + split_items_offset<Entry>());
  const uint32_t first = items[min(static_cast<int>(blockIdx.x) / kMergeUnits, kSplitMaxEntries - 1)];
  const int n_units = static_cast<int>(ws[0]) * kMergeUnits;
  // after a timeout the partials are incomplete: leave the output as it is
  if (err != nullptr && *reinterpret_cast<const volatile unsigned int*>(err) == kErrTimeout) return;
  const float* parts = reinterpret_cast<const float*>(split_area + split_partials_offset<Entry>());
  for (int unit = blockIdx.x; unit < n_units; unit += gridDim.x) {
    const int e = static_cast<int>(unit == static_cast<int>(blockIdx.x) ? first : items[unit / kMergeUnits]);
    const int t = unit % kMergeUnits / (kBlockM / kMergeRows);
    const int r0 = unit % (kBlockM / kMergeRows) * kMergeRows;
    const Entry en = reinterpret_cast<const Entry*>(split_area)[e];
    const TilePlace at = src.place(en, t);
    if (!at.exists || at.q0 + src.row(r0).token >= at.seg_end) continue;  // the whole CTA
    auto inside = [&](int r) { return at.q0 + src.row(r0 + r).token < at.seg_end; };
    auto part = [&](int ch) { return parts + (static_cast<size_t>(e + ch) * 2 + t) * kPartial<D>; };
    const int my_row = threadIdx.x / (D / 8), col = threadIdx.x % (D / 8) * 8;  // eight values of a row to a thread
    const bool mine = my_row < kMergeRows && inside(my_row);
    auto load = [&](int ch) {
      const float4* p = reinterpret_cast<const float4*>(part(ch) + static_cast<size_t>(r0 + my_row) * D + col);
      return Float8{p[0], p[1]};
    };
    constexpr int kAhead = 4;
    Float8 ahead[kAhead] = {};
    if (mine) {
#pragma unroll
      for (int ch = 0; ch < kAhead; ++ch)
        if (ch < en.chunks) ahead[ch] = load(ch);
    }
    __syncthreads();  // the previous unit's weights have been used
    {  // 16 lanes to a row
      const int r = threadIdx.x / 16, lane16 = threadIdx.x % 16;
      float mx = -INFINITY, den = 0.f;
      for (int ch = lane16; ch < en.chunks; ch += 16) {
        const float v = part(ch)[static_cast<size_t>(kBlockM) * D + r0 + r];
        s_w[r][ch] = v;
        mx = fmaxf(mx, v);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      const float base = mx == -INFINITY ? 0.f : mx;  // no chunk has weights: o is 0, the LSE -inf
      for (int ch = lane16; ch < en.chunks; ch += 16) den += __expf(s_w[r][ch] - base);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
      const float all = base + logf(den);
      for (int ch = lane16; ch < en.chunks; ch += 16) s_w[r][ch] = den == 0.f ? 0.f : __expf(s_w[r][ch] - all);
      if (lane16 == 0 && lse != nullptr && inside(r)) {
        const TileRow x = src.row(r0 + r);
        lse[static_cast<size_t>(at.head + x.head) * src.seg.capacity_q + at.q0 + x.token] = all;
      }
    }
    __syncthreads();
    if (mine) {
      const TileRow to = src.row(r0 + my_row);
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      auto add = [&](const Float8& v, float w) {
        acc[0] = fmaf(w, v.x.x, acc[0]);
        acc[1] = fmaf(w, v.x.y, acc[1]);
        acc[2] = fmaf(w, v.x.z, acc[2]);
        acc[3] = fmaf(w, v.x.w, acc[3]);
        acc[4] = fmaf(w, v.y.x, acc[4]);
        acc[5] = fmaf(w, v.y.y, acc[5]);
        acc[6] = fmaf(w, v.y.z, acc[6]);
        acc[7] = fmaf(w, v.y.w, acc[7]);
      };
#pragma unroll
      for (int ch = 0; ch < kAhead; ++ch)
        if (ch < en.chunks) add(ahead[ch], s_w[my_row][ch]);
#pragma unroll 4
      for (int ch = kAhead; ch < en.chunks; ++ch) add(load(ch), s_w[my_row][ch]);
      *reinterpret_cast<uint4*>(out + (static_cast<size_t>(at.q0 + to.token) * src.seg.num_q_heads + at.head + to.head) * D +
                                col) =
          make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]), pack_bf16x2(acc[4], acc[5]),
                     pack_bf16x2(acc[6], acc[7]));
    }
  }
}

}  // namespace
}  // namespace h3
