// kvq_roles.h -- the named barriers of the tile attention's softmax warps
// (kvq_tree.cu), for the kernel and for a host model of it.
//
// Every job, the eight warps of a slot vote (a reducing barrier) whether
// a reference must be raised, meet again on the vote's barrier if one must, and
// hand their weights over to the slot's first warp: seven arrive, the first
// waits.  While all waits for products succeed, nobody gets to the next vote before
// the first warp has taken the hand-over.  After a wait that ran out nothing
// else keeps a warp back, so the hand-over has a barrier of its own: on the vote's, a warp
// that has handed over would be counted again, with its next vote, in the same
// phase, results would differ between warps and some would wait for ever.
#pragma once

#ifdef __CUDACC__
#define KVQ_ROLES_HD __host__ __device__
#else
#define KVQ_ROLES_HD
#endif

namespace w4a8 {

constexpr int kBarQueries = 3;  // all softmax warps: the queries are in place
KVQ_ROLES_HD constexpr int bar_vote(int slot) { return 1 + slot; }
KVQ_ROLES_HD constexpr int bar_hand(int slot) { return 4 + slot; }

}  // namespace w4a8
