// Runs the recurrence's chain protocol (csrc/links.hpp) on the host, for every number
// of workgroups up to 40, and checks what orders its reads and writes.
//
// Each workgroup carries the set of chain-start reads that are known to be over
// when it acts: its own, and those of every workgroup whose word it has waited
// for, as that one knew them when it published.  The state that the chain ends
// with may be written over the start, so the last workgroup has to know all of
// them to be over.  A read counts as over at a publication only where the word is
// made of what was read: a load and a later store of one lane to different
// addresses keep no order of their own.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <set>
#include <utility>

#include "../differentiable_cholesky_amd/csrc/links.hpp"

namespace {

struct Word {
    bool there = false;
    float P = 0.f, Q = 0.f;
};

struct Trace {
    std::map<unsigned, Word> words;
    std::map<unsigned, std::set<unsigned>> over;     // by publisher: reads that its word follows
    std::map<unsigned, std::set<unsigned>> known;    // by workgroup, from the words it waited for
    std::set<unsigned> reads;                        // workgroups that read the start
};

struct Chain {
    Trace &t;
    unsigned self;
    float from;
    bool read = false;
    float start(int)
    {
        read = true;
        t.reads.insert(self);
        return from;
    }
    void publish(unsigned k, int, float P, float Q)
    {
        if (k != self || t.words[k].there)
            std::printf("workgroup %u publishes the word of %u, or a second time\n", self, k), std::exit(1);
        t.words[k] = {true, P, Q};
        t.over[k] = t.known[self];
        if (read)
            t.over[k].insert(self);
    }
    Word peek(unsigned k, int) { return t.words[k]; }
    float2 arrived(unsigned k, int, Word)
    {
        // workgroups start in order, so only an earlier one is certain to publish
        if (k >= self || !t.words[k].there)
            std::printf("workgroup %u waits for %u, which has not published\n", self, k), std::exit(1);
        t.known[self].insert(t.over[k].begin(), t.over[k].end());
        return make_float2(t.words[k].P, t.words[k].Q);
    }
};

// maps of small whole numbers, so that every order of composition is exact
float gate(unsigned k) { return k % 3 == 2 ? -1.f : 1.f; }
float input(unsigned k) { return (float)(k % 7) - 2.f; }

} // namespace

int main()
{
    for (unsigned chunks = 2; chunks <= 40; ++chunks) {
        Trace one, two;
        float want = 5.f;
        for (unsigned k = 0; k < chunks; ++k) {
            const float P[1] = {gate(k)}, Q[1] = {input(k)};
            float x[1], y[1];
            Chain a{one, k, 5.f}, b{two, k, 6.f};
            chol::state_before(a, k, chunks, P, Q, x);
            chol::state_before(b, k, chunks, P, Q, y);
            if (x[0] != want) {
                std::printf("%u of %u workgroups: state %g, not %g\n", k, chunks, x[0], want);
                return 1;
            }
            want = P[0] * want + Q[0];
            const bool depends = one.words[k].there && one.words[k].Q != two.words[k].Q;
            if (!depends) // nothing holds this workgroup's own read before its word
                one.over[k].erase(k);
        }
        std::set<unsigned> &known = one.known[chunks - 1];
        known.insert(chunks - 1); // it writes the end after what it read itself
        for (const unsigned k : one.reads)
            if (!known.count(k)) {
                std::printf("%u workgroups: the end is written while workgroup %u may still read the start\n", chunks, k);
                return 1;
            }
        if (one.reads.empty()) {
            std::printf("%u workgroups: nobody reads the start\n", chunks);
            return 1;
        }
    }
    std::printf("ordered\n");
    return 0;
}
