// How the roles of a persistent CTA go from one block of work to the next, when the next one is
// only known once it has been asked for (cluster launch control).  One role asks; every role
// takes the answer behind its own work on the block before.
//
// A wait may give up at any time, in any role, and the roles may learn of it at different times.
// Every role still has to leave its loop, and roles that meet at barriers have to leave it in the
// same pass:
//   - the asking role asks for block n + 1 only once every role has taken block n, so that no
//     answer changes before all have read it; when that wait gives up it asks no more;
//   - a role whose wait for the answer gives up takes "none" and does not count as having
//     taken it, so that nothing more is asked for;
//   - the members of a group that shares barriers take the same: what each took is put to the
//     vote at a barrier that they all reach in every pass, and one "none" is all of theirs.
//
// P: the role's primitives.  wait_free(n): block n has been taken by every role; wait_known(n):
// the answer to request n is there; both false once a wait has given up.  request(): ask;
// answer(): the block, or -1; taken(): this role has it.
#pragma once

#ifndef __CUDACC__
#define FBD_HD inline
#else
#define FBD_HD __device__ __forceinline__
#endif

namespace fbd {
namespace handover {

// Ask for the block after the n-th.  false: the asking role ends.
template <class P>
FBD_HD bool ask(const P& p, int n) {
  if (n > 0 && !p.wait_free(n - 1)) return false;
  p.request();
  return true;
}

// The block after the n-th, or -1.
template <class P>
FBD_HD int take(const P& p, int n) {
  if (!p.wait_known(n)) return -1;
  const int x = p.answer();
  p.taken();
  return x;
}

// `all`: a barrier of the group that says whether the argument is true for every member.
template <class All>
FBD_HD int agree(int x, const All& all) {
  return all(x >= 0) ? x : -1;
}

// Parity of the last phase that `fills` fills of a ring of `stages` have begun in stage s < fills:
// what a CTA that gave up waits for before it ends.
FBD_HD int last_phase(int fills, int stages, int s) { return ((fills - 1 - s) / stages) & 1; }

// Buffers handed from one role to another in turn, each with a barrier of its own that completes a phase a
// hand-over.  A parity tells two neighbouring phases apart, so a giver that may be `n` hand-overs ahead of a taker
// that has not yet looked needs n barriers, as it needs n buffers: on one barrier the second hand-over would
// look like none.  The buffer (and barrier) of hand-over k of n, and the parity of its wait.
FBD_HD int buffer_of(int k, int n) { return k % n; }
FBD_HD int parity_of(int k, int n) { return (k / n) & 1; }

}  // namespace handover
}  // namespace fbd
