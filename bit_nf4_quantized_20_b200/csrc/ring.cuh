// ring.cuh -- the loop of a TMA producer over a ring of shared-memory stages.
// Free of device code, so that it also compiles for the host.
#pragma once

#if defined(__CUDACC__)
#define QLORA_RING_FN __host__ __device__ __forceinline__
#else
#define QLORA_RING_FN inline
#endif

namespace qlora {

// Steps `first` .. `n` - 1 (the caller has issued those before, at most one
// round of the ring) through `stages` slots:
//   slot_free(s, parity)  bounded wait for slot s's last release; false: stop
//   issue(s, step)        arms the slot's barrier and starts its copies
//   landed(s, parity)     bounded wait for the copies of slot s
// A copy still in flight when its CTA leaves would write shared memory that
// another CTA may own by then.  The consumers see every copy land unless one of
// their waits runs out, which may happen at any time, after the last issue too:
// so the last round is waited for whatever ended the loop.  (Its barriers are
// not armed again, and the CTA waits for its consumers anyway.)  One of those
// waits running out has given the other copies its whole limit as well.
#if defined(__CUDACC__)
#pragma nv_exec_check_disable
#endif
template <class Free, class Issue, class Landed>
QLORA_RING_FN void feed_ring(int first, int n, int stages, const Free &slot_free, const Issue &issue,
                             const Landed &landed) {
  int issued = first, s = first == stages ? 0 : first;
  unsigned ph = first == stages ? 0u : 1u;   // parity of the slot's last release
  for (int st = first; st < n; ++st) {
    if (!slot_free(s, ph)) break;
    issue(s, st);
    issued = st + 1;
    if (++s == stages) {
      s = 0;
      ph ^= 1u;
    }
  }
  for (int st = issued > stages ? issued - stages : 0; st < issued; ++st)
    if (!landed(st % stages, static_cast<unsigned>(st / stages) & 1u)) break;
}

}  // namespace qlora
