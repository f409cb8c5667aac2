// The body of the decode kernel, with kTails of the shared-prefix kernel's tails
// and with kWindow of the windowed decode kernel (decode_kernel.cuh includes it in
// each of the functions).  In scope: Policy, Args, kTails, kWindow, a, tmk, tmv,
// base, units, others (the last two set with kTails).
    const int G = a.num_q_heads / a.num_kv_heads;
    const int Hc = a.heads_per_stage, R = a.warps_per_head, NC = a.consumer_warps;
    const int chunks = a.num_kv_heads / Hc;
    const int D = a.head_dim;
    const int half_bytes = Hc * a.block_size * D * dtype_bytes(a.kv_dtype);
    const SmemLayout L = smem_layout(a.stages, half_bytes, kTails || kWindow ? 2 * a.num_seqs : a.num_seqs, NC, R, G, D,
                                     a.block_size, Policy::kScratch);
    uint8_t* ring = base + L.ring;
    uint64_t* full = reinterpret_cast<uint64_t*>(base + L.full_bar);
    uint64_t* empty = reinterpret_cast<uint64_t*>(base + L.empty_bar);
    volatile int* abort = reinterpret_cast<volatile int*>(base + L.flags);
    int32_t* scan = reinterpret_cast<int32_t*>(base + L.scan);
    int32_t* cum = reinterpret_cast<int32_t*>(base + L.cum);
    int32_t* skip = cum + a.num_seqs + 1;  // kTails and kWindow only
    float* merge = reinterpret_cast<float*>(base + L.merge);

    const int tid = threadIdx.x;
    if (a.stages % R != 0) {  // see decode_plan: the ring must be a multiple of R
        if (tid == 0 && blockIdx.x == 0) raise_flag(a.status, kFlagBadPlan);
        return;
    }
    int P = a.num_ctas;
    if constexpr (kTails) {
        P = build_prefix<true, false>(a, chunks, cum, scan, skip, units);  // ends with __syncthreads
        if (static_cast<int>(blockIdx.x) >= P) {
            *others = true;
            return;
        }
    }
    if (tid == 0) {
        for (int st = 0; st < a.stages; ++st) {
            mbar_init(&full[st], 1);
            mbar_init(&empty[st], Hc);  // one arrival per head of the chunk
        }
        *abort = 0;
        fence_barrier_init();
        if constexpr (Policy::kTensor) {
            prefetch_tensor_map(&tmk);
            prefetch_tensor_map(&tmv);
        }
    }
    if constexpr (kTails) {
        __syncthreads();
    } else {
        // Everything above touches only this CTA's shared memory and parameters.
        // With early_reads the caller promises that the previous launch on the
        // stream writes neither the tables, the lengths nor the K/V cache, so the
        // prefix, the table entries and the first stages are fetched while that
        // launch finishes; everything else (q, the new rows, the workspace, the
        // outputs) is touched only after waiting for it.
        if (!a.early_reads) pdl_wait();
        build_prefix<false, kWindow>(a, chunks, cum, scan, skip, nullptr);  // ends with __syncthreads
    }
    const int64_t W = cum[a.num_seqs];
    const int start = static_cast<int>(static_cast<int64_t>(blockIdx.x) * W / P);
    const int end = static_cast<int>((static_cast<int64_t>(blockIdx.x) + 1) * W / P);
    const int warp = tid >> 5, lane = tid & 31;
    if (warp == 0 && start < end) {
        produce<Policy::kTensor, kTails, kWindow>(a, ring, full, empty, cum, skip, chunks, start, end, half_bytes, &tmk,
                                 &tmv, abort);
        return;
    }
    if (!kTails && a.early_reads) pdl_wait();
    // Global writes of the prologue, by the threads that are not producing.
    const int wt = start < end ? tid - 32 : tid;
    const int nwt = start < end ? static_cast<int>(blockDim.x) - 32 : static_cast<int>(blockDim.x);
    if constexpr (kTails) {
        for (int p = blockIdx.x + P * wt; p < a.num_seqs * chunks; p += P * nwt) {
            const int s = p / chunks;
            const int nbv = (cum[s + 1] - cum[s]) / chunks;
            a.tail_parts[p] = tail_parts_of(cum[s] + (p - s * chunks) * nbv + a.phantom, nbv - a.phantom, W, P);
        }
        // Sequences without prefix parts (the parts role speaks for the others).
        for (int p = blockIdx.x + P * wt; p < a.num_seqs * a.num_kv_heads; p += P * nwt)
            if (skip[p / a.num_kv_heads] == 0) a.prefix_parts[p] = make_int4(0, 0, 0, 0);
        if (warp > NC) return;  // the grid's blocks are as large as the parts role needs
    } else {
        if (blockIdx.x == 0 && !a.fused_reduce) {
            for (int s = wt; s <= a.num_seqs; s += nwt) a.cum[s] = cum[s];
        }
        // Sequences with no tokens: zero rows (fused merge) and slot -1 (CTA s mod P).
        for (int s = blockIdx.x; s < a.num_seqs; s += P) {
            if (cum[s + 1] != cum[s]) continue;
            if (a.slot_out && wt == 0) a.slot_out[s] = -1;
            if (!a.fused_reduce) continue;
            const int64_t o0 = static_cast<int64_t>(s) * a.num_q_heads * D;
            for (int e = wt; e < a.num_q_heads * D; e += nwt) store_out(a.out, o0 + e, 0.f, a.out_dtype);
        }
    }
    if (start >= end) return;

    const int w = warp - 1;
    const int hw = w % Hc;  // head within the chunk
    const int rr = w / Hc;  // replica among the R warps of that head
    float* scratch = Policy::kScratch
                         ? reinterpret_cast<float*>(base + L.scratch) +
                               w * ((a.block_size * G * 4 + 15) & ~15) / 4
                         : nullptr;
    Policy pol;
    typename Policy::State st;
    int seg = start;
    while (seg < end) {
        const int s = find_sequence(cum, a.num_seqs, seg);
        const int nbv = (cum[s + 1] - cum[s]) / chunks;  // the pair's items, phantoms included
        const int nb = nbv - a.phantom;                    // its blocks
        const int hc = (seg - cum[s]) / nbv;
        const int pair_a = cum[s] + hc * nbv;
        const int pair_b = pair_a + nbv;
        const int seg_end = min(pair_b, end);
        const int h = hc * Hc + hw;
        const int ctx = clamp_context(a, s, false) - (kTails ? skip[s] * a.block_size : 0);
        // kWindow: the first token of block j of the list, and what of the block is hidden.
        auto first_token = [&](int j) {
            if constexpr (kWindow) return (j + (j >= a.sink_blocks ? skip[s] : 0)) * a.block_size;
            return j * a.block_size;
        };
        auto hidden_in = [&](int j) {
            Hidden r{0, 0, 0.f};
            if constexpr (kWindow) {
                const int t0 = first_token(j);
                r.from = max(a.sinks - t0, 0);
                r.to = min(ctx - a.window - t0, a.block_size);
                r.lower = lower_of(ctx, a.window);
            }
            return r;
        };
        pol.begin(st, a, s, h, G);
        const int first = seg + (((rr - (seg - start)) % R) + R) % R;
        // Ring position of item `first` (item t = i - start sits in stage
        // t % stages, phase (t / stages) & 1); advanced by R per item below.
        int stage = (first - start) % a.stages;
        uint32_t phase = static_cast<uint32_t>((first - start) / a.stages) & 1u;
        for (int i = first; i < seg_end;) {
            // With a policy that takes two 16-token blocks at once, this warp
            // takes items i and i + R together when both belong to the run.
            // Waiting for the second while holding the first needs the
            // producer to have refilled stage (i + R) % stages, i.e. item
            // i + R - stages to be released: true when stages >= 2R.
            const int j = i - pair_a - a.phantom;  // block index; negative: a phantom item
            bool two = false;
            if constexpr (Policy::kPairs)
                two = a.block_size == 16 && i + R < seg_end && a.stages >= 2 * R && j >= 0;
            int stage2 = stage + R;  // R divides the ring size, so this wraps exactly at the end
            uint32_t phase2 = phase;
            if (stage2 >= a.stages) {
                stage2 -= a.stages;
                phase2 ^= 1u;
            }
            bool ok = mbar_wait_bounded(&full[stage], phase, abort, a.status);
            if (ok && two) ok = mbar_wait_bounded(&full[stage2], phase2, abort, a.status);
            if (ok && j >= 0) {
                const int n_valid = min(a.block_size, ctx - first_token(j));
                uint8_t* kt = ring + stage * 2 * half_bytes;
                bool patched = !kTails && !kWindow && a.k_new && j == nb - 1 && append_row(a, pol, kt, kt + half_bytes, s, h, hw, j, n_valid - 1);
                if constexpr (Policy::kPairs) {
                    if (two) {
                        const int j1 = j + R;
                        const int n1 = min(a.block_size, ctx - first_token(j1));
                        uint8_t* kt1 = ring + stage2 * 2 * half_bytes;
                        if (!kTails && !kWindow && a.k_new && j1 == nb - 1)
                            patched |= append_row(a, pol, kt1, kt1 + half_bytes, s, h, hw, j1, n1 - 1);
                        if constexpr (kWindow)
                            pol.template tile2<true>(st, a, kt, kt + half_bytes, n_valid, kt1, kt1 + half_bytes, n1,
                                                     hw, G, hidden_in(j), hidden_in(j1));
                        else
                            pol.tile2(st, a, kt, kt + half_bytes, n_valid, kt1, kt1 + half_bytes, n1, hw, G);
                    }
                }
                if constexpr (kWindow) {
                    if (!two)
                        pol.template tile<true>(st, a, kt, kt + half_bytes, hw, n_valid, G, scratch, hidden_in(j));
                } else {
                    if (!two) pol.tile(st, a, kt, kt + half_bytes, hw, n_valid, G, scratch);
                }
                if (patched) fence_proxy_async_smem();  // generic writes before the next TMA fill
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&empty[stage]);
                if (two) mbar_arrive(&empty[stage2]);
            }
            i += two ? 2 * R : R;
            stage = stage2;
            phase = phase2;
            if (two) {
                stage += R;
                if (stage >= a.stages) {
                    stage -= a.stages;
                    phase ^= 1u;
                }
            }
        }
        // The pair's blocks are its items [pair_r, pair_b) (phantoms first).
        // A segment holding none of them is not a part of the pair: it
        // writes nothing and counts no arrival (the same on every warp).
        const int pair_r = pair_a + a.phantom;
        const bool whole = !kTails && (pair_r >= start) && (pair_b <= end);
        const bool blocks = max(seg, pair_r) < seg_end;
        const int pair = s * chunks + hc;
        const int64_t sl = (static_cast<int64_t>(blockIdx.x + pair) * Hc + hw) * G;
        bool partial = false;  // this warp wrote the CTA's partial of (s, h)
        if (!blocks) {
        } else if (R == 1) {
            if (!*abort) {
                if (whole) {
                    pol.write_final(st, a, s, h, G);
                } else {
                    pol.write_partial(st, a, a.part_o + sl * D, a.part_ml + sl * 2, G);
                    partial = true;
                }
            }
        } else {
            // Merge the R warps of each head through shared memory.
            pol.write_state(st, a, merge + w * G * (D + 2), D + 2, G);
            named_barrier_sync(1, NC * 32);
            if (rr == 0 && !*abort) {
                combine_replicas(a, merge, hw, Hc, R, G, whole, s, h, a.part_o + sl * D,
                                 a.part_ml + sl * 2);
                partial = !whole;
            }
            named_barrier_sync(1, NC * 32);
        }
        if constexpr (!kTails) {
            // A split pair at the end of the range: once every consumer warp is
            // past its last stage, the ring's shared memory is free (the producer
            // issued nothing after the range's last item) and the merge may stage
            // the parts there, one slice a warp.
            float* staging = nullptr;
            int staging_floats = 0;
            if (R == 1 && a.fused_reduce && seg_end == end && !whole && blocks) {
                named_barrier_sync(1, NC * 32);
                staging_floats = (a.stages * 2 * half_bytes / NC / 4) & ~3;
                staging = reinterpret_cast<float*>(ring) + w * staging_floats;
            }
            if (partial && a.fused_reduce) {
                // The parts: the CTAs holding the pair's blocks.  With fewer
                // items than CTAs each block has its own CTA.
                const int ca = cta_of_item(pair_r, W, P);
                const int cb = cta_of_item(pair_b - 1, W, P);
                const int nparts = W >= P ? cb - ca + 1 : pair_b - pair_r;
                constexpr int T = Policy::kMaxThreads, DD = Policy::kD;
                switch (G) {
                    case 1:
                        merge_if_last<1, DD, merge_prefetch(1, DD, T)>(a, s, h, hw, pair, nparts, ca, cb, W,
                                                                      staging, staging_floats);
                        break;
                    case 2:
                        merge_if_last<2, DD, merge_prefetch(2, DD, T)>(a, s, h, hw, pair, nparts, ca, cb, W,
                                                                      staging, staging_floats);
                        break;
                    case 4:
                        merge_if_last<4, DD, merge_prefetch(4, DD, T)>(a, s, h, hw, pair, nparts, ca, cb, W,
                                                                      staging, staging_floats);
                        break;
                    default:
                        merge_if_last<8, DD, merge_prefetch(8, DD, T)>(a, s, h, hw, pair, nparts, ca, cb, W,
                                                                      staging, staging_floats);
                        break;
                }
            }
        }
        seg = seg_end;
    }
